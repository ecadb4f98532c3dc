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
    int out_dtype;
};

// One output: the bias, then one rounding to out's type.
__device__ __forceinline__ void store_int4(const Int4Args& a, int64_t row, int64_t col, float v)
{
    if (a.out_dtype == CK_OUT_FP32) {
        if (a.bias) v = v + bias_at<EPI_F32>(a.bias, col);
        static_cast<float*>(a.out)[row * a.ldo + col] = v;
        return;
    }
    uint16_t* const out = static_cast<uint16_t*>(a.out) + row * a.ldo + col;
    if (a.out_dtype == CK_OUT_FP16) {
        if (a.bias) v = v + bias_at<EPI_F16>(a.bias, col);
        *out = (uint16_t)(pack2<EPI_F16>(v, 0.0f) & 0xffffu);
    } else {
        if (a.bias) v = v + bias_at<EPI_BF16>(a.bias, col);
        *out = (uint16_t)(pack2<EPI_BF16>(v, 0.0f) & 0xffffu);
    }
}

// Few rows of x (up to 16).  Mathematics: for each group g of columns,
//   out[i, j] += s[j, g] (sum_t x[i, t] (16 + c[j, t]) - (16 + z[j, g]) X[i, g]),
//   X[i, g] = sum_t x[i, t],
// because 16 + c is one bit operation away from a code: the code's four bits
// are the upper mantissa bits of 16 in bf16 and in fp16 alike.  The products
// are exact in fp32, X comes from the same matrix cores (a product with
// ones), and the group's sum keeps about 3 bits less than one of c - z would:
// far below a 16-bit output's rounding, up to twice the error of a plain fp32
// product in an fp32 output.
//
// Bound: HBM; the weights are read once, 1 KiB at a time, in the order that
// ck_int4_pack laid them out in.  Each wave streams its part of K for NT row
// tiles of W through a ring of its own in LDS, filled by direct-to-LDS loads
// (W, scales and zeros, and x), so that no barrier and no register waits for
// them; the waves' sums meet in LDS at the end, in a fixed order.
//
// Products (16 x 16 x 32): x rows are the first operand and W rows the second,
// so lane 16 G + i holds column i.  Row j of a 16-row block of x sits at
// operand row 4 (j % 4) + j / 4, which puts it into register j / 4 of lanes
// G = j % 4: with up to 4 (8) rows only one (two) of the four accumulator
// registers are in use, and only those get the scales (MR).
//
// 1 x 28672 x 5376: groups of 128 16.2 us (4.9 TB/s), groups of 32 with zero
// points 20.0 us (4.6 TB/s): HBM, and the start and end of 256 to 896 blocks.
// 16384 x 4096, groups of 64 with zeros: 1 row 9.1 us, 4 9.6, 8 10.3, 16 12.9.
// 1 x 4096 x 4096: 4.0 us, where a launch of three blocks takes 3.1 us.
//
// mask and base are int4_mask and int4_base in registers of the two kinds that
// one and-or instruction takes (it has no room for constants).
template <int DT>
constexpr uint32_t int4_mask = DT == CK_DT_FP16 ? 0x03c003c0u : 0x00780078u;
template <int DT>
constexpr uint32_t int4_base = DT == CK_DT_FP16 ? 0x4c004c00u : 0x41804180u;      // 16, twice

template <int DT>
__device__ __forceinline__ v4i codes16(uint32_t w, uint32_t mask, uint32_t base)
{
    constexpr int up = DT == CK_DT_FP16 ? 6 : 3;                                  // bit of the code's place
    v4i r;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        r[p] = (int)(((4 * p <= up ? w << (up - 4 * p) : w >> (4 * p - up)) & mask) | base);
    return r;
}

template <int DT>
__device__ __forceinline__ float widen1(uint32_t bits16)
{
    return widen2<DT>(bits16).x;
}

template <int GS, int MR, int MB, int NT, int KW>
struct Int4Few {
    static constexpr int xl = MB * MR;                       // 1 KiB loads of x: four rows of 128
    static constexpr int slot = (NT + xl + 1) * 1024;        // W, x, then scales and zeros
    static constexpr int loads = NT + xl + 1;
    static constexpr int ring = KW * 2 * slot;               // more waves hide more than longer rings
    static constexpr int regs = NT * MB * MR;
    static constexpr int sums = KW * regs * 256;
    static_assert(sums <= ring && ring <= 163840 && loads < 64, "the ring, then the sums");
};

template <int DT, int GS, bool Z, int MR, int MB, int NT, int KW>
__global__ __launch_bounds__(64 * KW, 2) void int4_few_kernel(Int4Args a)
{
    using S = Int4Few<GS, MR, MB, NT, KW>;
    constexpr int XL = S::xl, L = S::loads;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[S::ring];
    const int lane = threadIdx.x & 63, G = lane >> 4, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tiles = (a.n + 15) / 16, tile0 = (int64_t)blockIdx.x * NT;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MB);
    const int rows = (int)min<int64_t>(a.m - m0, 16 * MB);
    const int cb = (int)(a.chunks * wave / KW), ce = (int)(a.chunks * (wave + 1) / KW), nc = ce - cb;

    const uint8_t* const xb = reinterpret_cast<const uint8_t*>(a.x + m0 * a.ldx);
    uint32_t x_off[XL], x_at[XL];                            // row, and byte of the chunk's 256
#pragma unroll
    for (int j = 0; j < XL; ++j) {
        const int row = 4 * j + G;
        x_off[j] = (uint32_t)(min(row, rows - 1) * a.ldx * 2);
        x_at[j] = (uint32_t)((i16 ^ (row & 15)) * 16);
    }
    // Scales: two lanes a tile and group; zeros from lane 32 on, one lane.
    const bool zl = Z && lane >= 32;
    const int su = zl ? lane - 32 : lane, per = zl ? 1 : 2;
    const int st = min(su / (GS * per), NT - 1), sg = su / per % GS;
    const int64_t stile = min(tile0 + st, tiles - 1);
    const uint8_t* const s_base = zl ? a.wz + stile * a.groups * 16
                                     : reinterpret_cast<const uint8_t*>(a.ws) + stile * a.groups * 32 + (su & 1) * 16;
    const uint32_t s_step = zl ? 16 : 32;
    const uint8_t* w_base[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) w_base[t] = a.w + min(tile0 + t, tiles - 1) * a.chunks * 1024;

    uint8_t* const my = ring + wave * (2 * S::slot);
    const uint32_t my_lds = lds_addr(my);
    auto issue = [&](int slot, int c) {
        const uint32_t dst = my_lds + slot * S::slot;
        const int64_t kc = cb + c;
#pragma unroll
        for (int t = 0; t < NT; ++t) dma16(reinterpret_cast<const int8_t*>(w_base[t] + kc * 1024), lane * 16, dst + t * 1024);
        const uint32_t left = (uint32_t)min<int64_t>(256, (a.k - kc * 128) * 2) - 16;   // past k: the last piece again
#pragma unroll
        for (int j = 0; j < XL; ++j)
            dma16(reinterpret_cast<const int8_t*>(xb + kc * 256), x_off[j] + min(x_at[j], left), dst + (NT + j) * 1024);
        const uint32_t g = (uint32_t)min<int64_t>(kc * GS + sg, a.groups - 1);
        dma16_at(s_base + (uint64_t)g * s_step, dst + (NT + XL) * 1024);
    };

    // x: operand row i of a 16-row block is row 4 (i % 4) + i / 4
    int x_rd[MB], x_sw[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int row = 16 * b + 4 * min(i16 & 3, MR - 1) + (i16 >> 2);
        x_rd[b] = NT * 1024 + row * 256;
        x_sw[b] = row & 15;
    }
    const uint32_t one2 = DT == CK_DT_FP16 ? 0x3c003c00u : 0x3f803f80u;
    const v4i one = {(int)one2, (int)one2, (int)one2, (int)one2};
    uint32_t mask = int4_mask<DT>, base16 = int4_base<DT>;
    asm volatile("" : "+v"(mask));
    asm volatile("" : "+s"(base16));
    const f32x4v zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    float tot[NT][MB][MR];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int r = 0; r < MR; ++r) tot[t][b][r] = 0.0f;

    if (nc > 0) issue(0, 0);
    if (nc > 1) issue(1, 1);
    auto consume = [&](int slot, int c) {
        uint8_t* const base = my + slot * S::slot;
        const int kleft = (int)min<int64_t>(128, a.k - (int64_t)(cb + c) * 128);
        if (kleft < 128) {                                   // x past k becomes zero
#pragma unroll
            for (int j = 0; j < XL; ++j)
                if ((i16 ^ ((4 * j + G) & 15)) * 8 >= kleft)
                    *reinterpret_cast<v4i*>(base + (NT + j) * 1024 + lane * 16) = v4i{0, 0, 0, 0};
        }
        v4i w[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t] = *reinterpret_cast<const v4i*>(base + t * 1024 + lane * 16);
#pragma unroll
        for (int g = 0; g < GS; ++g) {
            f32x4v acc[NT][MB], xs[MB];
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                xs[b] = zero4;
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t][b] = zero4;
            }
#pragma unroll
            for (int s = g * (4 / GS); s < (g + 1) * (4 / GS); ++s) {
                v4i x[MB];
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    x[b] = *reinterpret_cast<const v4i*>(base + x_rd[b] + (((4 * s + G) ^ x_sw[b]) << 4));
                    xs[b] = mfma16<DT>(x[b], one, xs[b]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const v4i wf = codes16<DT>((uint32_t)w[t][s], mask, base16);
#pragma unroll
                    for (int b = 0; b < MB; ++b) acc[t][b] = mfma16<DT>(x[b], wf, acc[t][b]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint8_t* const sp = base + (NT + XL) * 1024;
                const float sc = widen1<DT>(*reinterpret_cast<const uint16_t*>(sp + (t * GS + g) * 32 + i16 * 2));
                const float z = Z ? 16.0f + (float)sp[512 + (t * GS + g) * 16 + i16] : 24.0f;
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int r = 0; r < MR; ++r)
                        tot[t][b][r] = __builtin_fmaf(sc, __builtin_fmaf(-z, xs[b][r], acc[t][b][r]), tot[t][b][r]);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); // the slot is read
    };
    for (int c = 0; c < nc; ++c) {
        if (c + 1 < nc) wait_vmcnt<L>();                     // the next chunk is on its way
        else wait_vmcnt<0>();
        consume(c & 1, c);
        if (c + 2 < nc) issue(c & 1, c + 2);
    }

    // The waves' sums, over the rings, then in their order.
    __syncthreads();
    float* const red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int r = 0; r < MR; ++r) red[((wave * NT + t) * MB * MR + b * MR + r) * 64 + lane] = tot[t][b][r];
    __syncthreads();
    for (int o = threadIdx.x; o < S::regs * 64; o += 64 * KW) {
        const int l = o & 63, q = o >> 6, r = q % MR, b = q / MR % MB, t = q / (MR * MB);
        const int64_t col = (tile0 + t) * 16 + (l & 15);
        const int row = 16 * b + 4 * r + (l >> 4);
        if (col >= a.n || row >= rows) continue;
        float v = red[o];
#pragma unroll
        for (int w = 1; w < KW; ++w) v = v + red[w * S::regs * 64 + o];
        store_int4(a, m0 + row, col, v);
    }
}

// More rows of x (blocks of 16 MB = 32 or 64).  The same mathematics; now the
// waves of a block share x.  A wave has MB row blocks of x times NT row tiles
// of W; WN waves side by side make a team, and WK teams split K.  x comes
// into LDS in stages of 64 columns for every team (one in use and one on its
// way, one barrier a stage), W in chunks of 128 columns, two deep.  A wave
// takes a chunk's words and scales into registers at once; the next barrier
// frees the chunk's place.
//
// The sums X of x over a group are needed by every wave, but made by one:
// each wave forms those of its share of the row blocks and leaves them in
// LDS, and all waves take them off one stage later, after its barrier.
//
// Bound at 128 rows: the matrix cores (busy 22 % of the time), the vector unit
// (31 %: two fused multiply-adds per output and group, two operations per two
// codes) and the LDS reads of x (26 %, 1 KiB for NT products; two fifths of it
// bank conflicts) take turns rather than overlap, with two waves a SIMD that
// wait for a third of their time: 128 x 21504 x 5376 53 to 55 us, 550 TFLOP/s.
// Two blocks of four waves a CU overlap better than one of eight waves (64
// us).  At 32 rows HBM is as near: 32 x 21504 x 5376 23 us.  Rows past 128
// repeat the unpacking of W in every block of 64: 512 rows 175 us, 8192 rows
// 2.57 ms (740 TFLOP/s).
template <int GS, int MB, int NT, int WN, int WK>
struct Int4Many {
    static constexpr int waves = WN * WK;
    static constexpr int part = MB * 2048;                   // a team's stage of x
    static constexpr int stage = WK * part;
    static constexpr int slot = (NT + 1) * 1024;             // W, then scales and zeros
    static constexpr int wring = 2 * stage;
    static constexpr int xsum = wring + WN * WK * 2 * slot;  // [team][stage parity][group][16 blocks]
    static constexpr int hg = GS == 4 ? 2 : 1;               // groups per stage
    static constexpr int spare = xsum + WK * 2 * hg * MB * 64;   // where the lanes write that have no X
    static constexpr int bytes = spare + 1024;
    static constexpr int xl = MB * 2 / WN;                   // 1 KiB loads of x per wave and stage
    static constexpr int wl = NT + 1;                        // and of W per wave and chunk
    static constexpr int own = MB / WN;                      // row blocks whose X a wave makes
    static constexpr int regs = NT * MB * 4;
    static constexpr int sums = waves * regs * 256;
    static constexpr int total = bytes > sums ? bytes : sums;
    static_assert(MB % WN == 0 && total <= 163840, "sizes");
};

template <int DT, int GS, bool Z, int MB, int NT, int WN, int WK>
__global__ __launch_bounds__(64 * WN * WK, 2) void int4_many_kernel(Int4Args a)
{
    using S = Int4Many<GS, MB, NT, WN, WK>;
    constexpr int XL = S::xl, WL = S::wl, HG = S::hg;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::total];
    const int lane = threadIdx.x & 63, G = lane >> 4, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % WN, wk = wave / WN;
    const int64_t tiles = (a.n + 15) / 16, tile0 = ((int64_t)blockIdx.x * WN + wn) * NT;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MB);
    const int rows = (int)min<int64_t>(a.m - m0, 16 * MB);
    const int cb = (int)(a.chunks * wk / WK), ce = (int)(a.chunks * (wk + 1) / WK), nc = ce - cb;
    const int most = (int)((a.chunks + WK - 1) / WK);

    // x: load j of a team's stage copies rows 8 j + lane / 8, 16-byte piece
    // lane % 8, pieces exchanged by xor so that 16 rows' same piece lie apart
    const uint8_t* const xb = reinterpret_cast<const uint8_t*>(a.x + m0 * a.ldx);
    uint32_t x_off[XL], x_at[XL];
#pragma unroll
    for (int j = 0; j < XL; ++j) {
        const int row = 8 * (wn + WN * j) + (lane >> 3);
        x_at[j] = (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
        x_off[j] = (uint32_t)(min(row, rows - 1) * a.ldx * 2) + x_at[j];
    }
    const uint32_t lds0 = lds_addr(lds);
    auto issue_x = [&](int h, int o) {
        const int64_t k0 = (int64_t)cb * 128 + h * 64;
        const uint32_t dst = lds0 + o * S::stage + wk * S::part;
        if (k0 + 64 <= a.k) {
#pragma unroll
            for (int j = 0; j < XL; ++j)
                dma16(reinterpret_cast<const int8_t*>(xb + k0 * 2), x_off[j], dst + (wn + WN * j) * 1024);
        } else {                                             // past k: the row's last piece again, zeroed before use
            const int64_t base = k0 >= a.k ? (a.k - 8) * 2 : k0 * 2;
            const uint32_t cap = (uint32_t)(a.k * 2 - base) - 16;
#pragma unroll
            for (int j = 0; j < XL; ++j)
                dma16(reinterpret_cast<const int8_t*>(xb + base), x_off[j] - x_at[j] + min(x_at[j], cap), dst + (wn + WN * j) * 1024);
        }
    };
    // W, scales (two lanes a tile and group) and zeros (one lane, from 32 on)
    const bool zl = Z && lane >= 32;
    const int su = zl ? lane - 32 : lane, per = zl ? 1 : 2;
    const int st = min(su / (GS * per), NT - 1), sg = su / per % GS;
    const int64_t stile = min(tile0 + st, tiles - 1);
    const uint8_t* const s_base = zl ? a.wz + stile * a.groups * 16
                                     : reinterpret_cast<const uint8_t*>(a.ws) + stile * a.groups * 32 + (su & 1) * 16;
    const uint32_t s_step = zl ? 16 : 32;
    const uint8_t* w_base[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) w_base[t] = a.w + min(tile0 + t, tiles - 1) * a.chunks * 1024;
    uint8_t* const my = lds + S::wring + (wk * WN + wn) * (2 * S::slot);
    const uint32_t my_lds = lds_addr(my);
    auto issue_w = [&](int c) {
        const uint32_t dst = my_lds + (c & 1) * S::slot;
        const int64_t kc = cb + c;
#pragma unroll
        for (int t = 0; t < NT; ++t)
            dma16(reinterpret_cast<const int8_t*>(w_base[t] + kc * 1024), lane * 16, dst + t * 1024);
        const uint32_t g = (uint32_t)min<int64_t>(kc * GS + sg, a.groups - 1);
        dma16_at(s_base + (uint64_t)g * s_step, dst + NT * 1024);
    };

    const uint32_t one2 = DT == CK_DT_FP16 ? 0x3c003c00u : 0x3f803f80u;
    const v4i one = {(int)one2, (int)one2, (int)one2, (int)one2};
    const f32x4v zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t mask = int4_mask<DT>, base16 = int4_base<DT>;
    asm volatile("" : "+v"(mask));
    asm volatile("" : "+s"(base16));
    f32x4v tot[NT][MB], acc[NT][GS == 1 ? MB : 1], xacc[S::own];   // acc, xacc: a group longer than a stage
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < MB; ++b) tot[t][b] = zero4;
    v4i w[NT];                                               // the chunk's words
    float sc[NT][GS], sz[NT][GS];                            // its scales, and scales times (16 + zero)
    float sz_was[NT][HG];                                    // those of the X in LDS (none yet)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int g = 0; g < HG; ++g) sz_was[t][g] = 0.0f;
    for (int i = threadIdx.x; i < WK * 2 * HG * MB * 4; i += 64 * S::waves)
        reinterpret_cast<f32x4v*>(lds + S::xsum)[i] = zero4;
    f32x4v* const xsum = reinterpret_cast<f32x4v*>(lds + S::xsum) + wk * (2 * HG * MB * 4);
    const uint32_t x_wr = i16 == 0 ? S::xsum + (wk * 2 * HG * MB * 4 + G) * 16 : S::spare + lane * 16;
    auto take_off = [&](int o, bool now) {                   // the X of the stage before, of parity o
        if (!now) return;
#pragma unroll
        for (int g = 0; g < HG; ++g)
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const f32x4v x = xsum[((o * HG + g) * MB + b) * 4 + G];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) tot[t][b][r] = __builtin_fmaf(-sz_was[t][g], x[r], tot[t][b][r]);
            }
    };
    // x's row in a 16-row block for this lane's operand row, and its two pieces
    const int x_row = 4 * (i16 & 3) + (i16 >> 2), x_sw = (x_row >> 1) & 7;
    const int x_rd[2] = {x_row * 128 + ((G ^ x_sw) << 4), x_row * 128 + (((4 + G) ^ x_sw) << 4)};
    auto half = [&](int c, auto odd) {
        constexpr int O = decltype(odd)::value ? 1 : 0;
        const uint8_t* const xs = lds + O * S::stage + wk * S::part;
        if (O == 0) {
            const uint8_t* const base = my + (c & 1) * S::slot;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                w[t] = *reinterpret_cast<const v4i*>(base + t * 1024 + lane * 16);
#pragma unroll
                for (int g = 0; g < GS; ++g) {
                    sc[t][g] = widen1<DT>(*reinterpret_cast<const uint16_t*>(base + NT * 1024 + (t * GS + g) * 32 + i16 * 2));
                    const float z = Z ? 16.0f + (float)base[NT * 1024 + 512 + (t * GS + g) * 16 + i16] : 24.0f;
                    sz[t][g] = sc[t][g] * z;
                }
            }
        }
        // x of the next stage goes where the stage before this one was, and
        // after an even stage W of two chunks on where this chunk's was
        if (O == 0 || c + 1 < nc) issue_x(2 * c + O + 1, 1 - O);
        if (O == 1 && c + 2 < nc) issue_w(c + 2);
        take_off(GS > 1 ? 1 - O : 0, GS > 1 || O == 0);
        constexpr int SG = 2 / HG;                           // steps of 32 columns per group of this stage
        // X of this wave's row blocks
#pragma unroll
        for (int i = 0; i < S::own; ++i) {
            const int b = wn + WN * i;
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                f32x4v sum = GS == 1 && O == 1 ? xacc[i] : zero4;
#pragma unroll
                for (int s = g * SG; s < (g + 1) * SG; ++s)
                    sum = mfma16<DT>(*reinterpret_cast<const v4i*>(xs + b * 2048 + x_rd[s]), one, sum);
                if (GS == 1 && O == 0) xacc[i] = sum;
                else *reinterpret_cast<f32x4v*>(lds + x_wr + (i16 == 0 ? (((GS > 1 ? O : 0) * HG + g) * MB + b) * 64 : 0)) = sum;
            }
        }
        v4i wf[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s) wf[t][s] = codes16<DT>((uint32_t)w[t][2 * O + s], mask, base16);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            v4i x[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) x[s] = *reinterpret_cast<const v4i*>(xs + x_rd[s] + b * 2048);
#pragma unroll
            for (int g = 0; g < HG; ++g) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f32x4v sum = GS == 1 && O == 1 ? acc[t][GS == 1 ? b : 0] : zero4;
#pragma unroll
                    for (int s = g * SG; s < (g + 1) * SG; ++s) sum = mfma16<DT>(x[s], wf[t][s], sum);
                    if (GS == 1 && O == 0) {
                        acc[t][GS == 1 ? b : 0] = sum;
                        continue;
                    }
                    const float scale = sc[t][GS == 4 ? 2 * O + g : GS == 2 ? O : 0];
#pragma unroll
                    for (int r = 0; r < 4; ++r) tot[t][b][r] = __builtin_fmaf(scale, sum[r], tot[t][b][r]);
                }
            }
            // Left alone, the compiler moves the scaling of all products to
            // where the sums are used next, past the stage's end, and runs
            // out of registers on the way.
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (GS > 1 || O == 1) asm volatile("" : "+v"(tot[t][b]));
                else asm volatile("" : "+v"(acc[t][GS == 1 ? b : 0]));
            }
        }
        if (GS > 1 || O == 1) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int g = 0; g < HG; ++g) sz_was[t][g] = sz[t][GS == 4 ? 2 * O + g : GS == 2 ? O : 0];
        }
    };
    const bool tail = a.k % 128 != 0;
    auto clear_tail = [&](int h, int o) {                    // x past k in a landed stage becomes zero
        const int64_t left = a.k - ((int64_t)cb * 128 + h * 64);
        if (left < 64) {
#pragma unroll
            for (int j = 0; j < XL; ++j)
                if ((int)x_at[j] >= 2 * left)
                    *reinterpret_cast<v4i*>(lds + o * S::stage + wk * S::part + (wn + WN * j) * 1024 + lane * 16) = v4i{0, 0, 0, 0};
        }
    };
    // The end of a stage: this wave's loads of x of the next one have landed,
    // and after an odd stage those of the next chunk of W; only the W that was
    // issued last, after that x, may be on its way.
    auto close = [&](int c, auto odd) {
        constexpr int O = decltype(odd)::value ? 1 : 0;
        if (O == 1 && c + 2 < nc) wait_vmcnt<WL>();
        else wait_vmcnt<0>();
        if (tail) clear_tail(2 * c + O + 1, 1 - O);
        __syncthreads();
    };

    if (nc > 0) {
        issue_x(0, 0);
        issue_w(0);
        if (nc > 1) issue_w(1);
    }
    if (nc > 1) wait_vmcnt<WL>();                            // x of stage 0 and W of chunk 0
    else wait_vmcnt<0>();
    if (tail) clear_tail(0, 0);
    __syncthreads();
    for (int c = 0; c < nc; ++c) {
        half(c, BoolTag<false>{});
        close(c, BoolTag<false>{});
        half(c, BoolTag<true>{});
        close(c, BoolTag<true>{});
    }
    for (int c = nc; c < most; ++c) {                        // a team with a chunk less than another
        __syncthreads();
        __syncthreads();
    }
    if (nc > 0) take_off(GS > 1 ? 1 : 0, true);

    // The teams' sums, over everything, then in their order.
    __syncthreads();
    float* const red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[(wave * S::regs + (t * MB + b) * 4 + r) * 64 + lane] = tot[t][b][r];
    __syncthreads();
    for (int o = threadIdx.x; o < WN * S::regs * 64; o += 64 * S::waves) {
        const int l = o & 63, q = (o >> 6) % S::regs, wv = (o >> 6) / S::regs, r = q & 3, b = (q >> 2) % MB, t = (q >> 2) / MB;
        const int64_t col = (((int64_t)blockIdx.x * WN + wv) * NT + t) * 16 + (l & 15);
        const int row = 16 * b + 4 * r + (l >> 4);
        if (col >= a.n || row >= rows) continue;
        float v = red[o];
#pragma unroll
        for (int k = 1; k < WK; ++k) v = v + red[o + k * WN * S::regs * 64];
        store_int4(a, m0 + row, col, v);
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

// The kernel for a call, and what a block of it covers.
struct Int4Plan {
    const void* fn;
    int tiles, rows, waves;
};

template <int DT, int GS, bool Z>
Int4Plan int4_plan_gs(int64_t m, int64_t n, int64_t chunks)
{
#define CK_INT4_FEW(MR, MB, NT, KW) \
    Int4Plan{reinterpret_cast<const void*>(&int4_few_kernel<DT, GS, Z, MR, MB, NT, KW>), NT, 16 * MB, KW}
#define CK_INT4_MANY(MB, NT, WN, WK, ONE, TWO)                                                    \
    {{reinterpret_cast<const void*>(&int4_many_kernel<DT, GS, Z, MB, NT, WN, WK>), NT * WN, 16 * MB, \
      WN * WK}, WK, ONE, TWO}
    // Few rows: eight waves, four from 8193 columns on, and above 20480 columns
    // eight waves of two row tiles, by the number of blocks (16 columns a row
    // tile).  1 row, groups of 128, eight waves / four / eight of two tiles, us:
    //   4096 x 4096   4.4  5.6  5.2      20480 x 4096  11.0  10.4  12.5
    //   8192 x 4096   6.0  6.7  6.6      21504 x 5376  14.9  15.1  14.1
    //   10240 x 4096  7.4  7.4  8.2      24576 x 5376  15.4  15.4  14.7
    //   16384 x 4096 10.1  8.9  10.1     28672 x 5376  18.0  18.4  17.6
    // Groups of 32 follow them, but for equal times of the last two columns at
    // 28672.  k does not enter: with 1024 columns two tiles are up to 8 % slower
    // there than four waves would be (28672: 6.6 against 6.1).
    const bool wide = n > 20480;
    if (m <= 4) return wide ? CK_INT4_FEW(1, 1, 2, 8) : n > 8192 ? CK_INT4_FEW(1, 1, 1, 4) : CK_INT4_FEW(1, 1, 1, 8);
    if (m <= 8) return wide ? CK_INT4_FEW(2, 1, 2, 8) : n > 8192 ? CK_INT4_FEW(2, 1, 1, 4) : CK_INT4_FEW(2, 1, 1, 8);
    if (m <= 16) return wide ? CK_INT4_FEW(4, 1, 2, 8) : n > 8192 ? CK_INT4_FEW(4, 1, 1, 4) : CK_INT4_FEW(4, 1, 1, 8);
    // More rows: a round of 256 blocks, one a CU, takes about 2 us and ONE /
    // 100 us for each chunk of a team; where two blocks fit a CU's LDS, a
    // round of up to 512 takes TWO / 100 us a chunk.  (Fitted to group 128 at
    // 17 to 128 rows of 4096 x 4096, 8192 x 4096, 16384 x 4096, 21504 x 5376 and
    // 28672 x 5376; groups of 32 take 1.5 times as long in the same order.)
    // The least sum wins: 128 rows of 21504 x 5376 take 66, 52, 62 and 70 us
    // with blocks of 64, 96 and 128 columns of four waves and 128 columns of
    // eight, of 16384 x 4096 34, 42, 36 and 30 us.
    struct Choice { Int4Plan plan; int teams, one, two; };
    const Choice upto32[] = {CK_INT4_MANY(2, 2, 1, 8, 110, 0), CK_INT4_MANY(2, 2, 2, 4, 110, 0), CK_INT4_MANY(2, 4, 2, 4, 190, 0)};
    const Choice more[] = {CK_INT4_MANY(4, 1, 2, 4, 175, 0), CK_INT4_MANY(4, 2, 2, 2, 155, 190), CK_INT4_MANY(4, 3, 2, 2, 180, 240),
                           CK_INT4_MANY(4, 4, 2, 2, 205, 290), CK_INT4_MANY(4, 2, 2, 4, 230, 0), CK_INT4_MANY(4, 4, 2, 4, 335, 0)};
    const Choice* const from = m <= 32 ? upto32 : more;
    const int count = m <= 32 ? 3 : 6;
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < count; ++i) {
        const Choice& c = from[i];
        const int64_t blocks = cdiv(cdiv(n, 16), c.plan.tiles) * cdiv(m, c.plan.rows), each = cdiv(chunks, c.teams);
        const int64_t round = c.two ? 2 * kNumCUs : kNumCUs, rest = blocks % round;
        const int64_t full = 200 + each * (c.two ? c.two : c.one);
        const int64_t time = blocks / round * full + (rest > kNumCUs ? full : rest > 0 ? 200 + each * c.one : 0);
        if (time < least) least = time, best = i;
    }
    return from[best].plan;
#undef CK_INT4_MANY
#undef CK_INT4_FEW
}

template <int DT, bool Z>
Int4Plan int4_plan_z(int64_t m, int64_t n, int64_t chunks, int64_t group)
{
    return group == 32   ? int4_plan_gs<DT, 4, Z>(m, n, chunks)
           : group == 64 ? int4_plan_gs<DT, 2, Z>(m, n, chunks)
                         : int4_plan_gs<DT, 1, Z>(m, n, chunks);
}

Int4Plan int4_plan(int dtype, bool zeros, int64_t m, int64_t n, int64_t chunks, int64_t group)
{
    if (dtype == CK_DT_FP16) return zeros ? int4_plan_z<CK_DT_FP16, true>(m, n, chunks, group) : int4_plan_z<CK_DT_FP16, false>(m, n, chunks, group);
    return zeros ? int4_plan_z<CK_DT_BF16, true>(m, n, chunks, group) : int4_plan_z<CK_DT_BF16, false>(m, n, chunks, group);
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
    if (!grid_ok(blocks, 256)) return fail(CK_ERR_UNSUPPORTED, "too many blocks");
    if ((s = check_device()) != CK_OK) return s;
    void* kargs[] = {&a};
    s = launch(reinterpret_cast<const void*>(&int4_pack_kernel), (unsigned)blocks, 256, kargs, stream, "int4_pack");
    return s == CK_OK ? ok() : s;
}

extern "C" ck_status ck_int4_linear(const ck_int4_args* args, hipStream_t stream)
{
    if (!args) return fail(CK_ERR_INVALID_ARG, "NULL args");
    const ck_int4_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.out_dtype != CK_OUT_BF16 && p.out_dtype != CK_OUT_FP16 && p.out_dtype != CK_OUT_FP32)
        return fail(CK_ERR_INVALID_ARG, "bad out_dtype");
    if (p.m < 0) return fail(CK_ERR_INVALID_ARG, "negative size");
    ck_status s = check_int4_sizes(p.n, p.k, p.group);
    if (s != CK_OK) return s;
    if (p.m == 0 || p.n == 0) return ok();
    if (!p.out) return fail(CK_ERR_INVALID_ARG, "NULL out");
    if (p.m > 1 && p.ldo < p.n) return fail(CK_ERR_INVALID_ARG, "ldo smaller than n");
    if (p.k > 0) {
        if (!p.x || !p.w || !p.w_scale) return fail(CK_ERR_INVALID_ARG, "NULL x, w or w_scale");
        if (p.m > 1 && p.ldx < p.k) return fail(CK_ERR_INVALID_ARG, "ldx smaller than k");
        if ((p.m > 1 && p.ldx % 8 != 0) || !aligned(p.x, 16))
            return fail(CK_ERR_UNSUPPORTED, "x rows must start 16 bytes apart (ldx %% 8 == 0)");
    }
    const int esz = p.out_dtype == CK_OUT_FP32 ? 4 : 2;
    if (!aligned(p.w, 16) || !aligned(p.w_scale, 16) || !aligned(p.w_zero, 16) || !aligned(p.out, esz) ||
        (p.bias && !aligned(p.bias, esz)))
        return fail(CK_ERR_UNSUPPORTED, "misaligned w, w_scale, w_zero, bias or out");
    // 32-bit offsets of a block's rows of x
    if (p.m > 1 && 256 * p.ldx >= (int64_t(1) << 31))
        return fail(CK_ERR_UNSUPPORTED, "rows of x too long for 32-bit offsets");
    const Int4Plan plan = int4_plan(p.dtype, p.w_zero != nullptr, p.m, p.n, cdiv(p.k, 128), p.group);
    const int64_t bx = cdiv(cdiv(p.n, 16), plan.tiles), by = cdiv(p.m, plan.rows);
    if (by > 65535 || !grid_ok(bx, 64 * plan.waves)) return fail(CK_ERR_UNSUPPORTED, "too many rows or columns");
    if ((s = check_device()) != CK_OK) return s;
    Int4Args a{(const uint16_t*)p.x, p.w, p.w_scale, p.w_zero, p.bias, p.out, p.ldx, p.ldo, p.m, p.n, p.k,
               cdiv(p.k, 128), cdiv(p.k, p.group), p.out_dtype};
    void* kargs[] = {&a};
    hipError_t e = hipLaunchKernel(plan.fn, dim3((unsigned)bx, (unsigned)by), dim3(64 * plan.waves), kargs, 0, stream);
    if (e != hipSuccess) return fail(CK_ERR_HIP, "int4_linear launch: %s", hipGetErrorString(e));
    return ok();
}
