// lora_add.hip -- y + s (x A^T) B^T with a low-rank adapter for every row.
//
// Mathematics.  For a row i with adapter t: v = x[i] A_t^T (rank sums over k),
// then out[i] = y[i] + (s_t v) B_t^T.  Both products run on the matrix cores
// (16 x 16 x 32) with fp32 sums.  v stays 32 bits: it enters the second product
// in 16-bit parts, three of bf16 (2^-24 of it), or two of fp16 after a power of
// two that brings the row's largest to [2^13, 2^14) (2^-22 of it, or 2^-38 of the
// largest).
//
// Bound: HBM, by the adapters that a decode batch asks for or by y of a
// prompt, and the launches of small calls.  Rows are taken 64 at a time, those
// with the same adapter together whatever their order, so an adapter is read
// once for its rows; a row without one is copied.
//   - Up to kLoraRows rows, a block has one adapter of a group of up to 64 rows and a
//     slice of the columns.  Where A is small every block makes v by itself, in
//     the same launch: A comes from L2 then, once for each slice.
//   - Otherwise a first launch makes v, with k split over blocks where there
//     are few of them (their parts are added in order by the second).
//   - More rows are those of prompts: a block goes through the adapters of its
//     rows in turn, mostly one, and holds a piece of B for 64 rows.

struct LoraArgs {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    const int32_t* ids;
    const void* y;
    void* out;
    float* v;                            // [ksplits][m][vstride], of the first launch
    int64_t ldx, ldy, ldo, a_stride, b_stride, m;
    int n, k, rank, adapters;
    int vstride, ksplits, slices, slice; // slice: columns of one
    int turn;                            // where B's pieces are in LDS
    int copy, wide;                      // rows without an adapter are copied; 16-byte accesses of y and out
};

constexpr int kLoraRows = 512;           // rows up to which every adapter of 64 rows has its own blocks
constexpr int kLoraWaves = 8;            // of a block that makes v

template <int N> struct IntTag { static constexpr int value = N; };

// The next adapter among up to 64 rows, each lane with its row's id, and the
// rows that have it; `left`: those still to come.
__device__ __forceinline__ uint64_t lora_members(uint64_t& left, int ids, int& id)
{
    id = __builtin_amdgcn_readlane(ids, __builtin_ctzll(left));
    const uint64_t members = __ballot(ids == id) & left;
    left &= ~members;
    return members;
}

// The rows of a block: `left` of them have an adapter (`without`: those that
// have none).  With units > 0 the block has the unit-th adapter alone, and of the
// others every units-th row.
struct LoraRows {
    int64_t r0;
    int count, ids;                      // this lane's row's id
    uint64_t left, without;

    __device__ __forceinline__ LoraRows(const LoraArgs& a, int64_t block, int group, int units)
    {
        const int lane = threadIdx.x & 63;
        int unit = units > 0 ? (int)(block % units) : 0;
        r0 = (units > 0 ? block / units : block) * group;
        count = (int)min<int64_t>(group, a.m - r0);
        ids = lane < count ? a.ids[r0 + lane] : -1;
        left = __ballot(ids >= 0 && ids < a.adapters);
        without = __ballot(lane < count && (units == 0 || lane % units == unit)) & ~left;
        int id;
        for (; unit > 0 && left; --unit) lora_members(left, ids, id);
        if (units > 0 && left) {
            uint64_t rest = left;
            left = lora_members(rest, ids, id);
        }
    }
};

// The members in order: lane p gets the p-th one's row.
__device__ __forceinline__ int lora_places(uint64_t members)
{
    const int lane = threadIdx.x & 63, before = __popcll(members & ((1ull << lane) - 1));
    return __builtin_amdgcn_ds_permute((members >> lane & 1 ? before : __popcll(members) + lane - before) * 4, lane);
}

// d[0] of a quad's first lane + d[1] of its second + d[2] of its third + d[3] of
// its fourth, in all four.
__device__ __forceinline__ float quad_diagonal(const f32x4v& d)
{
    const int t0 = __builtin_amdgcn_update_dpp(0, __float_as_int(d[0]), 0x00, 0xf, 0xf, true);
    const int t1 = __builtin_amdgcn_update_dpp(0, __float_as_int(d[1]), 0x55, 0xf, 0xf, true);
    const int t2 = __builtin_amdgcn_update_dpp(0, __float_as_int(d[2]), 0xaa, 0xf, 0xf, true);
    const int t3 = __builtin_amdgcn_update_dpp(0, __float_as_int(d[3]), 0xff, 0xf, 0xf, true);
    return (__int_as_float(t0) + __int_as_float(t1)) + (__int_as_float(t2) + __int_as_float(t3));
}

// The first product, 16 ranks from rank0 on of 4 XG rows, over steps s0 .. s1 - 1
// of 128 columns.  A load of 16 bytes a lane costs as many cycles as the 64-byte
// segments that each four lanes in a row touch, so such four take 64 bytes of
// a row of A or x, which makes them different operand rows: row 4 a + b of the
// first operand is piece b (8 columns) of A's row a, column 4 c + b of the second
// piece b of x's row c, and where the two b agree the product is a part of v, four
// of which add up to it.  (With operand rows that are A's and x's the loads took
// three times as long.)  Lane 16 G + 4 c + b ends up with ranks rank0 + 4 q + G of
// row 4 g + c in v[g][q], for every b.  The code is short on purpose: a call runs
// most of it once or twice, and it comes from a cold instruction cache at some
// 10 cycles an instruction (64 ranks a wave instead of 16 took 13 us for 8).
// xo: the rows' byte offsets from xb, with this lane's columns of 128.
template <int DT, int XG>
__device__ __forceinline__ void lora_shrink(const LoraArgs& a, const uint16_t* xb, const uint32_t (&xo)[XG], const uint16_t* wb,
                                            int rank0, int s0, int s1, float (&v)[XG][4])
{
    constexpr int U = XG == 4 ? 2 : 4;                       // steps whose loads go out together
    const int lane = threadIdx.x & 63;
    const int at = (lane >> 4) * 32 + (lane & 3) * 8;        // this lane's columns of 128
    const int last = (a.rank - rank0) / 4 - 1;               // of the groups of four ranks
    const uint32_t wo = (uint32_t)(((lane >> 2) & 3) * a.k + at) * 2;
    const char* const x = reinterpret_cast<const char*>(xb);
    const char* w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = reinterpret_cast<const char*>(wb + (int64_t)(rank0 + 4 * min(q, last)) * a.k);
    f32x4v acc[XG][4];
#pragma unroll
    for (int g = 0; g < XG; ++g)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[g][q] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
    auto run = [&](int s, auto count) {
        constexpr int N = decltype(count)::value;
        v4i xs[N][XG], ws[N][4];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            uint32_t off = (s + u) * 256;
            if (N == 1) off = min(off + 2 * at, (uint32_t)(2 * a.k - 16)) - 2 * at;      // past the end the row's last piece again, times zeros
#pragma unroll
            for (int g = 0; g < XG; ++g) xs[u][g] = *reinterpret_cast<const v4i*>(x + (xo[g] + off));
#pragma unroll
            for (int q = 0; q < 4; ++q) ws[u][q] = *reinterpret_cast<const v4i*>(w[q] + (wo + off));
        }
        if (N == 1 && s * 128 + at >= a.k) {
#pragma unroll
            for (int g = 0; g < XG; ++g) xs[0][g] = v4i{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int g = 0; g < XG; ++g) acc[g][q] = mfma16<DT>(ws[u][q], xs[u][g], acc[g][q]);
    };
    const int full = min(s1, a.k / 128);
    int s = s0;
    for (; s + U <= full; s += U) run(s, IntTag<U>{});
    for (; s < s1; ++s) run(s, IntTag<1>{});
#pragma unroll
    for (int g = 0; g < XG; ++g)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[g][q] = quad_diagonal(acc[g][q]);
}

// How a block's waves share the first product: a wave has 16 ranks, and the
// waves with the same ones each a part of k.
struct LoraShare {
    int groups, mine, part, parts;       // groups of 16 ranks at a time (a power of two), this wave's; its part of k
    __device__ __forceinline__ LoraShare(int rank, int wave, int split, int splits)
    {
        groups = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : kLoraWaves;
        mine = wave & (groups - 1);
        parts = kLoraWaves / groups * splits;
        part = split * (kLoraWaves / groups) + wave / groups;
    }
    __device__ __forceinline__ int begin(int steps, int more) const { return (int)((int64_t)steps * (part + more) / parts); }
};

// The rows that a lane's x are, as byte offsets: row 4 g + c of 16 from place t0
// on, the last one again past the end.
template <int XG>
__device__ __forceinline__ void lora_x(const LoraArgs& a, int places, int t0, int rows, uint32_t (&xo)[XG])
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int g = 0; g < XG; ++g)
        xo[g] = (uint32_t)(__shfl(places, min(t0 + 4 * g + ((lane >> 2) & 3), rows - 1)) * (uint32_t)a.ldx + (lane >> 4) * 32 + (lane & 3) * 8) * 2;
}

// The first launch: v of a group of rows, over one part of k, for the rows of an
// adapter 16 at a time, and four where there are no more (16 rows cost their
// loads, but one pass over A; 256 rows of 4 adapters in a row, 4096 columns, rank
// 16: 12.5 us, and 31.8 four at a time).
template <int DT>
__global__ __launch_bounds__(64 * kLoraWaves, 4) void lora_shrink_kernel(LoraArgs a, int group, int units)
{
    constexpr int NW = kLoraWaves;
    __shared__ float red[NW][16][20];                        // [wave][row][rank]
    const int tid = threadIdx.x, lane = tid & 63, G = lane >> 4, c = (lane >> 2) & 3;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int split = blockIdx.x % a.ksplits;
    LoraRows r(a, blockIdx.x / a.ksplits, group, units);
    const LoraShare share(a.rank, wave, split, a.ksplits);
    const int steps = (a.k + 127) / 128, s0 = share.begin(steps, 0), s1 = share.begin(steps, 1);
    while (r.left) {
        int id;
        const uint64_t members = lora_members(r.left, r.ids, id);
        const int rows = __popcll(members), places = lora_places(members);
        auto some = [&](int t0, auto size) {                 // 4 XG rows from place t0 on
            constexpr int XG = decltype(size)::value;
            uint32_t xo[XG];
            lora_x<XG>(a, places, t0, rows, xo);
            for (int rank0 = 0; rank0 < a.rank; rank0 += 16 * share.groups) {
                if (rank0 + 16 * share.mine < a.rank) {
                    float v[XG][4];
                    lora_shrink<DT, XG>(a, a.x + r.r0 * a.ldx, xo, a.a + id * a.a_stride, rank0 + 16 * share.mine, s0, s1, v);
                    if ((lane & 3) == 0) {
#pragma unroll
                        for (int g = 0; g < XG; ++g)
#pragma unroll
                            for (int q = 0; q < 4; ++q) red[wave][4 * g + c][4 * q + G] = v[g][q];
                    }
                }
                __syncthreads();
                for (int e = tid; e < 64 * XG * share.groups; e += 64 * NW) {
                    const int rr = e & 15, i = (e >> 4) % (4 * XG), g = e / (64 * XG), k = rank0 + 16 * g + rr;
                    const int row = __shfl(places, min(t0 + i, rows - 1));
                    if (t0 + i < rows && k < a.rank) {
                        float sum = red[g][i][rr];
                        for (int x = g + share.groups; x < NW; x += share.groups) sum = sum + red[x][i][rr];
                        a.v[((int64_t)split * a.m + r.r0 + row) * a.vstride + k] = sum;
                    }
                }
                __syncthreads();
            }
        };
        for (int t0 = 0; t0 < rows;) {
            if (rows - t0 > 4) {
                some(t0, IntTag<4>{});
                t0 += 16;
            } else {
                some(t0, IntTag<1>{});
                t0 += 4;
            }
        }
    }
}

// A lane's 16 of 64 columns of a row of y: the 16-byte pieces G, G + 4 and so on,
// at `off` and every 64 bytes on.
template <int OUT>
struct LoraRow {
    static constexpr int E = OUT == CK_OUT_FP32 ? 4 : 8, B = 16 / E;         // columns of a piece, bytes of a column
    static constexpr int T = OUT == CK_OUT_FP16 ? CK_DT_FP16 : CK_DT_BF16;
    v4i y[B];

    __device__ __forceinline__ void load(const char* base, uint32_t off)
    {
#pragma unroll
        for (int j = 0; j < B; ++j) y[j] = *reinterpret_cast<const v4i*>(base + (off + 64 * j));
    }
    // out = y + d
    __device__ __forceinline__ void store(char* base, uint32_t off, const f32x4v (&d)[4])
    {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            v4i o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (OUT == CK_OUT_FP32) {
                    o[i] = __float_as_int(__int_as_float(y[j][i]) + d[j][i]);
                } else {
                    const float2 f = widen2<T>((uint32_t)y[j][i]);
                    o[i] = (int)narrow2<T>(f.x + d[2 * j + i / 2][i % 2 * 2], f.y + d[2 * j + i / 2][i % 2 * 2 + 1]);
                }
            }
            *reinterpret_cast<v4i*>(base + (off + 64 * j)) = o;
        }
    }
    // One column.
    __device__ static __forceinline__ void add(const char* y, char* out, float d)
    {
        if constexpr (OUT == CK_OUT_FP32)
            *reinterpret_cast<float*>(out) = *reinterpret_cast<const float*>(y) + d;
        else
            *reinterpret_cast<uint16_t*>(out) = (uint16_t)narrow2<T>(widen2<T>(*reinterpret_cast<const uint16_t*>(y)).x + d, 0.0f);
    }
};

// The second product, or all of it (FUSED: v is made here), for up to `blocks`
// blocks of 16 rows at a time.  A wave has 64 columns at a time, as four tiles
// whose operand rows are such columns that lane 16 G + i ends up with whole
// 16-byte pieces of row i, G and every fourth one on: a load or store of y has 64
// bytes of each row.
template <int DT, int OUT, bool FUSED, int PR>
__global__ __launch_bounds__(64 * (FUSED ? 8 : 4), FUSED ? 4 : 3) void lora_expand_kernel(LoraArgs a, int units, int blocks)
{
    constexpr int PARTS = DT == CK_DT_FP16 ? 2 : 3, NW = FUSED ? kLoraWaves : 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, G = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slice = blockIdx.x % a.slices;
    const int c0 = slice * a.slice, c1 = min(a.n, c0 + a.slice);
    LoraRows r(a, blockIdx.x / a.slices, 64, units);
    if (a.copy) {                                            // rows without an adapter, as they are
        for (; r.without; r.without &= r.without - 1) {
            const int64_t row = r.r0 + __builtin_ctzll(r.without);
            for (int c = c0 + tid; c < c1; c += 64 * NW) {
                if constexpr (OUT == CK_OUT_FP32) static_cast<uint32_t*>(a.out)[row * a.ldo + c] = static_cast<const uint32_t*>(a.y)[row * a.ldy + c];
                else static_cast<uint16_t*>(a.out)[row * a.ldo + c] = static_cast<const uint16_t*>(a.y)[row * a.ldy + c];
            }
        }
    }
    const int steps = (a.rank + 31) / 32;                    // of the second product's sum
    v4i* const frags = reinterpret_cast<v4i*>(lds);          // [blocks][PARTS][steps][64]: v, its second operand
    float* const back = reinterpret_cast<float*>(frags + blocks * PARTS * steps * 64);   // [16 blocks] powers of two that v was divided by
    uint32_t* const tops = reinterpret_cast<uint32_t*>(back + 16 * blocks);              // [16 blocks] fp16: the rows' largest
    // Two values of a row, of ranks k and k + 1 (k even), in their 16-bit parts.
    auto put = [&](int i, int k, float x, float z) {
        uint32_t* const to = reinterpret_cast<uint32_t*>(frags + (i / 16 * PARTS * steps + k / 32) * 64 + k / 8 % 4 * 16 + i % 16) + k % 8 / 2;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            const uint32_t h = narrow2<DT>(x, z);
            const float2 f = widen2<DT>(h);
            to[p * steps * 256] = h;
            x -= f.x;
            z -= f.y;
        }
    };
    auto lift = [&](int i) { return 14 - __builtin_amdgcn_frexp_expf(__uint_as_float(tops[i])); };   // of a finite largest > 0
    // B of 64 columns comes in 16-byte pieces in their order, up to 8 PR ranks at
    // a time, and goes through this wave's part of LDS into the operands' order
    // (rows an odd number of pieces apart).
    v4i* const turn = reinterpret_cast<v4i*>(lds + a.turn) + wave * 64 * (PR | 1);
    float* const line = reinterpret_cast<float*>(lds + a.turn + NW * 64 * (PR | 1) * 16) + wave * 64;
    int cols[4];                                             // the column of this lane's operand row of each tile, of 64
#pragma unroll
    for (int t = 0; t < 4; ++t)
        cols[t] = OUT == CK_OUT_FP32 ? 16 * t + i16 : 32 * (t >> 1) + 8 * (i16 >> 2) + 4 * (t & 1) + (i16 & 3);
    while (r.left) {
        int id;
        const uint64_t members = lora_members(r.left, r.ids, id);
        const int rows = __popcll(members), places = lora_places(members);
        const float scale = a.scale ? a.scale[id] : 1.0f;
        const uint16_t* const bp = a.b + id * a.b_stride;
        const char* const yb = static_cast<const char*>(a.y) + r.r0 * a.ldy * LoraRow<OUT>::B;
        char* const ob = static_cast<char*>(a.out) + r.r0 * a.ldo * LoraRow<OUT>::B;
        // pieces of ranks 8 PR h and on of columns c and on
        const int prow = lane / PR, piece = lane % PR;
        auto load_b = [&](v4i (&w)[PR], int c, int h) {
            if (c >= a.n || 8 * (PR * h + piece) >= a.rank) return;      // (a wave may have no columns)
            const uint16_t* const from = bp + (int64_t)c * a.rank + 8 * PR * h;
            const int rest = a.n - 1 - c;                    // the last column again past the end
#pragma unroll
            for (int j = 0; j < PR; ++j) {
                const int row = j * (64 / PR) + prow;
                w[j] = *reinterpret_cast<const v4i*>(reinterpret_cast<const char*>(from) + (uint32_t)((rest >= 63 ? row : min(row, rest)) * a.rank + 8 * piece) * 2);
            }
        };
        auto turn_b = [&](const v4i (&w)[PR]) {
#pragma unroll
            for (int j = 0; j < PR; ++j) turn[(j * (64 / PR) + prow) * (PR | 1) + piece] = w[j];
        };
        v4i w[PR];
#pragma unroll
        for (int j = 0; j < PR; ++j) w[j] = v4i{0, 0, 0, 0};
        load_b(w, c0 + wave * 64, 0);                        // on its way while v is made
        for (int t0 = 0; t0 < rows; t0 += 16 * blocks) {
            const int here = min(16 * blocks, rows - t0);
            using Row = LoraRow<OUT>;
            Row io;                                          // y of the first rows and columns, on its way too
            auto load_y = [&](int c, int b) {                // this lane's row of the b-th 16, whole pieces only
                if (!a.wide || c + 64 > a.n || 16 * b + i16 >= here) return;
                const int row = __shfl(places, t0 + 16 * b + i16);
                io.load(yb + (int64_t)c * Row::B, (uint32_t)row * (uint32_t)a.ldy * Row::B + 16 * G);
            };
            load_y(c0 + wave * 64, 0);
            // v with the adapter's scale, four ranks of a row a thread; zeros past the last rank
            float val[4][4];
            int count = 0;
            if (DT == CK_DT_FP16 && tid < 16 * blocks) tops[tid] = 0;
            if constexpr (FUSED) {
                float* const red = reinterpret_cast<float*>(tops + 16);      // [waves][16 rows][16 ranks + 4]
                const LoraShare share(a.rank, wave, 0, 1);
                const int all = (a.k + 127) / 128, s0 = share.begin(all, 0), s1 = share.begin(all, 1), cc = (lane >> 2) & 3;
                for (int g0 = 0; g0 < here; g0 += 4) {
                    uint32_t xo[1];
                    lora_x<1>(a, places, t0 + g0, rows, xo);
                    float part[1][4];
                    if (16 * share.mine < a.rank)
                        lora_shrink<DT, 1>(a, a.x + r.r0 * a.ldx, xo, a.a + id * a.a_stride, 16 * share.mine, s0, s1, part);
                    if ((lane & 3) == 0) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) red[(wave * 16 + g0 + cc) * 20 + 4 * q + G] = part[0][q];
                    }
                }
                __syncthreads();
                const int i = tid >> 3, k = tid % 8 * 4;
                if (i < here) {
                    f32x4v sum = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (k < a.rank)
                        for (int x = k / 16; x < NW; x += share.groups) sum = sum + *reinterpret_cast<const f32x4v*>(red + (x * 16 + i) * 20 + k % 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) val[0][j] = sum[j] * scale;
                    count = 1;
                }
            } else {
                // up to 1024 of them (16 rows of 256 ranks, or 64 of 64): four a thread, all loads together
                f32x4v sum[4];
                const int per = 8 * steps, total = (here + 15) / 16 * 16 * per;
                count = (total - tid + 64 * NW - 1) / (64 * NW);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = tid + j * 64 * NW, i = q / per, k = (q - i * per) * 4;
                    const int64_t at = r.r0 + __shfl(places, min(t0 + i, rows - 1));
                    sum[j] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
                    if (j < count && i < here && k < a.rank) {
                        const float* const p = a.v + at * a.vstride + k;
                        for (int x = 0; x < a.ksplits; x += 4) {
                            f32x4v f[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                f[y] = x + y < a.ksplits ? *reinterpret_cast<const f32x4v*>(p + (int64_t)(x + y) * a.m * a.vstride)
                                                         : f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int y = 0; y < 4; ++y) sum[j] = sum[j] + f[y];
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) val[j][x] = sum[j][x] * scale;
            }
            const int per = FUSED ? 8 : 8 * steps;
            if constexpr (DT == CK_DT_FP16) {
                if (!FUSED) __syncthreads();                 // tops is cleared
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float top = 0.0f;
#pragma unroll
                    for (int x = 0; x < 4; ++x) top = fmaxf(top, __builtin_fabsf(val[j][x]));
                    if (j < count && top > 0.0f && top < INFINITY) atomicMax(&tops[(tid + j * 64 * NW) / per], __float_as_uint(top));
                }
                __syncthreads();
                if (tid < here) back[tid] = tops[tid] ? __builtin_amdgcn_ldexpf(1.0f, -lift(tid)) : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= count) break;
                const int q = tid + j * 64 * NW, i = q / per, k = (q - i * per) * 4;
                if constexpr (DT == CK_DT_FP16) {
                    const int e = tops[i] ? lift(i) : 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) val[j][x] = __builtin_amdgcn_ldexpf(val[j][x], e);
                }
                put(i, k, val[j][0], val[j][1]);
                put(i, k + 2, val[j][2], val[j][3]);
            }
            __syncthreads();
            for (int c = c0 + wave * 64; c < c1; c += 64 * NW) {
                // the columns that follow, or the first ones again for the next rows
                const int next = c + 64 * NW < c1 ? c + 64 * NW : c0 + wave * 64;
                const int groups = (a.rank + 8 * PR - 1) / (8 * PR);
                if (groups == 1) {
                    turn_b(w);
                    load_b(w, next, 0);
                }
#pragma unroll 1
                for (int b = 0; 16 * b < here; ++b) {
                    f32x4v acc[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[t] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
                    for (int h = 0; h < groups; ++h) {
                        if (groups > 1) {
                            turn_b(w);
                            load_b(w, h + 1 < groups || 16 * (b + 1) < here ? c : next, h + 1 < groups ? h + 1 : 0);
                        }
#pragma unroll
                        for (int s = 0; s < (PR + 3) / 4; ++s) {
                            const int k = PR * h + 4 * s;        // pieces before
                            if (8 * k >= a.rank) break;
                            // (pieces past the last rank meet zeros of v: any that is there does)
                            const int have = 8 * (k + G) < a.rank ? 4 * s + G : 0;
                            v4i f[4];
#pragma unroll
                            for (int t = 0; t < 4; ++t) f[t] = turn[cols[t] * (PR | 1) + have];
#pragma unroll
                            for (int p = 0; p < PARTS; ++p) {
                                const v4i y = frags[((b * PARTS + p) * steps + k / 4) * 64 + lane];
#pragma unroll
                                for (int t = 0; t < 4; ++t) acc[t] = mfma16<DT>(f[t], y, acc[t]);
                            }
                        }
                    }
                    if constexpr (DT == CK_DT_FP16) {
                        const float up = back[16 * b + i16];
#pragma unroll
                        for (int t = 0; t < 4; ++t) acc[t] = acc[t] * up;
                    }
                    if (a.wide && c + 64 <= a.n) {
                        const int row = __shfl(places, min(t0 + 16 * b + i16, rows - 1));
                        if (16 * b + i16 < here) io.store(ob + (int64_t)c * Row::B, (uint32_t)row * (uint32_t)a.ldo * Row::B + 16 * G, acc);
                    } else {                                 // a row's 64 columns, one a lane
                        for (int i = 0; i < min(16, here - 16 * b); ++i) {
                            if (i16 == i) {
#pragma unroll
                                for (int t = 0; t < 4; ++t)
                                    *reinterpret_cast<f32x4v*>(line + (OUT == CK_OUT_FP32 ? 16 * t + 4 * G : 32 * (t >> 1) + 8 * G + 4 * (t & 1))) = acc[t];
                            }
                            const int64_t row = __shfl(places, t0 + 16 * b + i);
                            const float d = line[lane];
                            if (c + lane < a.n) Row::add(yb + (row * a.ldy + c + lane) * Row::B, ob + (row * a.ldo + c + lane) * Row::B, d);
                        }
                    }
                    if (16 * (b + 1) < here) load_y(c, b + 1);
                    else if (c + 64 * NW < c1) load_y(c + 64 * NW, 0);
                }
            }
            __syncthreads();
        }
    }
}

namespace {

bool lora_sizes_ok(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    return m >= 0 && n >= 0 && k >= 0 && m <= (1 << 24) && n <= (1 << 24) && k <= (1 << 24) && k % 8 == 0 && rank >= 8 &&
           rank <= 256 && rank % 8 == 0;
}

struct LoraPlan {
    bool each, fused;                                        // an adapter a block; one launch
    int blocks;                                              // row blocks that the second product has in LDS
    int64_t group, ksplits, bytes;                           // of the first launch: rows of a block, parts of k
};

// Up to kLoraRows rows an adapter has blocks of its own: rows of 48 adapters in any
// order (4096 x 4096, rank 16) take 35 us so at 512 rows and 125 one after the
// other, at 1024 rows 59 and 111; but rows of one adapter, or few, in a row 14 us
// either way at 512, and 25 to 96 or 14 at 1024.  One launch for both products where
// A is small (16 rows; rank 16, k 8192: 8.0 us in one, 10.0 in two; k 16384: 10.0 and
// 9.5) and rows are few (61 rows of 48 adapters 16.0 and 20.0 us; 512 rows of 4
// adapters 45 and 33).
LoraPlan lora_plan(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    LoraPlan p{};
    p.each = m <= kLoraRows;
    p.fused = p.each && rank <= 32 && rank * k <= 131072 && m <= 64;
    p.blocks = p.fused || rank > 128 ? 1 : rank > 64 ? 2 : 4;    // within 64 KiB
    p.group = m <= 64 ? 64 : 16;
    const int64_t units = p.each ? std::min<int64_t>(m, 16) : cdiv(m, p.group);
    p.ksplits = std::max<int64_t>(1, std::min<int64_t>(cdiv(kNumCUs, std::max<int64_t>(units, 1)), cdiv(k * std::min<int64_t>(cdiv(rank, 16), kLoraWaves), 128 * 2 * kLoraWaves)));
    if (!p.fused) p.bytes = p.ksplits * m * rank * 4;
    return p;
}

template <int DT, int OUT>
const void* lora_expand_out(bool fused, int64_t rank)
{
    if (fused)
        return rank <= 16 ? reinterpret_cast<const void*>(&lora_expand_kernel<DT, OUT, true, 2>)
                          : reinterpret_cast<const void*>(&lora_expand_kernel<DT, OUT, true, 4>);
    return rank <= 16   ? reinterpret_cast<const void*>(&lora_expand_kernel<DT, OUT, false, 2>)
           : rank <= 32 ? reinterpret_cast<const void*>(&lora_expand_kernel<DT, OUT, false, 4>)
                        : reinterpret_cast<const void*>(&lora_expand_kernel<DT, OUT, false, 8>);
}

template <int DT>
const void* lora_expand_fn(int out_dtype, bool fused, int64_t rank)
{
    return out_dtype == CK_OUT_FP32   ? lora_expand_out<DT, CK_OUT_FP32>(fused, rank)
           : out_dtype == CK_OUT_FP16 ? lora_expand_out<DT, CK_OUT_FP16>(fused, rank)
                                      : lora_expand_out<DT, CK_OUT_BF16>(fused, rank);
}

}  // namespace

extern "C" int64_t ck_lora_add_workspace(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    return lora_sizes_ok(m, n, k, rank) ? lora_plan(m, n, k, rank).bytes : -1;
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
    if (p.m > 1 && p.out == p.y && p.ldo != p.ldy) return fail(CK_ERR_INVALID_ARG, "out is y with another ld");
    if (p.adapters > 0) {
        if (!p.b || (p.k > 0 && (!p.x || !p.a))) return fail(CK_ERR_INVALID_ARG, "NULL x, a or b");
        if (p.k > 0 && p.m > 1 && p.ldx < p.k) return fail(CK_ERR_INVALID_ARG, "ldx smaller than k");
        if (p.adapters > 1 && (p.a_stride < p.rank * p.k || p.b_stride < p.rank * p.n))
            return fail(CK_ERR_INVALID_ARG, "a_stride or b_stride smaller than an adapter");
        if ((p.k > 0 && p.m > 1 && p.ldx % 8 != 0) || (p.adapters > 1 && (p.a_stride % 8 != 0 || p.b_stride % 8 != 0)) ||
            !aligned(p.x, 16) || !aligned(p.a, 16) || !aligned(p.b, 16))
            return fail(CK_ERR_UNSUPPORTED, "rows of x and adapters must start 16 bytes apart");
    }
    // 32-bit offsets of 64 rows
    if (p.m > 1 && ((p.adapters > 0 && p.k > 0 && p.ldx > (1 << 24) + 128) || p.ldy > (1 << 24) + 128 || p.ldo > (1 << 24) + 128))
        return fail(CK_ERR_UNSUPPORTED, "rows of x, y or out more than 2^24 + 128 elements apart");
    const int esz = p.out_dtype == CK_OUT_FP32 ? 4 : 2;
    if (!aligned(p.y, esz) || !aligned(p.out, esz) || !aligned(p.ids, 4) || !aligned(p.scale, 4))
        return fail(CK_ERR_UNSUPPORTED, "misaligned y, out, ids or scale");
    const LoraPlan plan = lora_plan(p.m, p.n, p.k, p.rank);
    if (plan.bytes > 0 && (!p.workspace || p.workspace_bytes < plan.bytes))
        return fail(CK_ERR_INVALID_ARG, "the workspace needs %lld bytes", (long long)plan.bytes);
    if (!aligned(p.workspace, 256)) return fail(CK_ERR_UNSUPPORTED, "misaligned workspace");
    ck_status s = check_device();
    if (s != CK_OK) return s;
    LoraArgs a{(const uint16_t*)p.x, (const uint16_t*)p.a, (const uint16_t*)p.b, p.scale, p.ids, p.y, p.out, (float*)p.workspace,
               p.ldx, p.ldy, p.ldo, p.a_stride, p.b_stride, p.m, (int)p.n, (int)p.k, (int)p.rank,
               (int)(p.k > 0 ? p.adapters : 0), (int)p.rank, (int)plan.ksplits, 1, 0, 0, p.out != p.y, 0};
    a.wide = aligned(p.y, 16) && aligned(p.out, 16) && p.ldy * esz % 16 == 0 && p.ldo * esz % 16 == 0;
    const bool f16 = p.dtype == CK_DT_FP16;
    // As many blocks for 64 rows as they can have adapters, or one.
    int group = (int)plan.group, units = plan.each ? (int)std::max<int64_t>(1, std::min(std::min<int64_t>(64, p.m), p.adapters)) : 0;
    const int64_t per64 = cdiv(p.m, 64) * std::max(units, 1);
    if (!plan.fused && a.adapters > 0) {
        int few = std::min(group, units);
        void* kargs[] = {&a, &group, &few};
        const int64_t blocks = cdiv(p.m, plan.group) * std::max(few, 1) * plan.ksplits;
        const void* fn = f16 ? reinterpret_cast<const void*>(&lora_shrink_kernel<CK_DT_FP16>)
                             : reinterpret_cast<const void*>(&lora_shrink_kernel<CK_DT_BF16>);
        if ((s = launch(fn, (unsigned)blocks, 64 * kLoraWaves, kargs, stream, "lora_shrink")) != CK_OK) return s;
    }
    // Column slices, of whole rounds of a block's waves: as many blocks as give every CU two.
    const int64_t waves = plan.fused ? 8 : 4;
    const int64_t turns = cdiv(p.n, 64 * waves);             // of all columns
    a.slice = (int)(cdiv(turns, std::min(cdiv(2 * kNumCUs, per64), turns)) * 64 * waves);
    a.slices = (int)cdiv(p.n, a.slice);
    int held = plan.blocks;
    const int64_t parts = f16 ? 2 : 3, steps = cdiv(p.rank, 32);
    a.turn = (int)(held * parts * steps * 1024 + 128 * held + (plan.fused ? waves * 64 * 20 : 0));
    const size_t lds = a.turn + waves * 256 + waves * 64 * 16 * ((p.rank <= 16 ? 2 : p.rank <= 32 ? 4 : 8) + 1);
    const void* fn = f16 ? lora_expand_fn<CK_DT_FP16>(p.out_dtype, plan.fused, p.rank) : lora_expand_fn<CK_DT_BF16>(p.out_dtype, plan.fused, p.rank);
    void* kargs[] = {&a, &units, &held};
    const int64_t blocks = per64 * a.slices;
    hipError_t e = hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(64 * (unsigned)waves), kargs, lds, stream);
    if (e != hipSuccess) return fail(CK_ERR_HIP, "lora_add launch: %s", hipGetErrorString(e));
    return ok();
}
