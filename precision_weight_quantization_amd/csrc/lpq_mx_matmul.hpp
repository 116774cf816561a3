// Products of microscaled matrices.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

// y[m, n] = sum over k of a[m, k] * b[n, k], both operands with a power-of-two
// scale per 32 elements along k.  The matrix instruction
// v_mfma_scale_f32_16x16x128_f8f6f4 takes E4M3 or E2M1 values with a UE8M0
// byte for each lane's row and 32-element block, so the codes and scales go
// into it as they are stored.
//
// Operand layout (checked lane by lane): lane l holds row l % 16, and with g =
// l / 16: of an E2M1 operand the 16 bytes of elements 32g to 32g + 31; of an
// E4M3 operand two 16-byte pieces, elements 16g to 16g + 15 and 64 + 16g to 64
// + 16g + 15; the scale of block g in its scale register's low byte.  Result
// register r of lane l is row 4 * (l / 16) + r of the first operand, row l % 16
// of the second.  The weights (b) are the first operand, so that a lane holds 4
// neighbouring columns of y.
//
// Sums: the instruction adds 128 products and the accumulator in one step.
// E2M1 products are summed exactly; with an E4M3 operand it aligns them to the
// largest and drops what lies about 2^-16 below it (relative error of a sum
// over normal data 4e-6 to 3e-5, for any length), which is why a result with
// an E4M3 operand is offered in BF16 only.
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct MatmulArgs {
    const uint8_t *a, *ae;   // [M, K], scales [M, K / 32]
    const uint8_t *b, *be;   // [N, K], scales [N, K / 32]
    void* y;                 // [M, N] BF16 or FP32
    int32_t M, N, K;
    int32_t f32;             // y is FP32
};

// A lane's part of one 16-row, 128-element operand.
template <bool FP4>
struct Frag {
    v4u lo, hi;       // hi: E4M3 only
    uint32_t scale;
};

template <bool FP4>
constexpr int row_bytes(int k) {
    return FP4 ? k / 2 : k;
}

template <bool FP4>
__device__ __forceinline__ v8i frag_regs(const Frag<FP4>& f) {
    if constexpr (FP4) return v8i{(int)f.lo.x, (int)f.lo.y, (int)f.lo.z, (int)f.lo.w, 0, 0, 0, 0};
    else return v8i{(int)f.lo.x, (int)f.lo.y, (int)f.lo.z, (int)f.lo.w, (int)f.hi.x, (int)f.hi.y, (int)f.hi.z, (int)f.hi.w};
}

template <bool FP4A, bool FP4B>
__device__ __forceinline__ v4f mfma(const Frag<FP4A>& a, const Frag<FP4B>& b, v4f c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag_regs(a), frag_regs(b), c, FP4A ? 4 : 0, FP4B ? 4 : 0, 0,
                                                            (int)a.scale, 0, (int)b.scale);
}

// The lane's part of elements k0 to k0 + 127 from its row in memory; zeros with
// scale 1 past K and for a lane without a row.
template <bool FP4>
__device__ __forceinline__ Frag<FP4> load_frag(const uint8_t* row, const uint8_t* scales, bool in, int k0, int K, int g) {
    Frag<FP4> f;
    if constexpr (FP4) {
        f.lo = in && k0 + 32 * g < K ? load<false>(reinterpret_cast<const v4u*>(row + k0 / 2 + 16 * g)) : v4u{};
    } else {
        f.lo = in && k0 + 16 * g < K ? load<false>(reinterpret_cast<const v4u*>(row + k0 + 16 * g)) : v4u{};
        f.hi = in && k0 + 64 + 16 * g < K ? load<false>(reinterpret_cast<const v4u*>(row + k0 + 64 + 16 * g)) : v4u{};
    }
    f.scale = in && k0 + 32 * g < K ? load_u8(scales + k0 / 32 + g) : 127u;
    return f;
}

// Four neighbouring results of row m from column n on.
__device__ __forceinline__ void store_y4(const MatmulArgs& A, int64_t m, int n, v4f c) {
    const int64_t at = m * A.N + n;
    if (A.N % 4 == 0) {   // n is a multiple of 4: whole and aligned
        if (A.f32) store<false>(reinterpret_cast<v4f*>(static_cast<float*>(A.y) + at), c);
        else store<false>(reinterpret_cast<v2u*>(static_cast<uint16_t*>(A.y) + at), v2u{bf16x2(c[0], c[1]), bf16x2(c[2], c[3])});
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; r++) {
        if (n + r >= A.N) break;
        if (A.f32) static_cast<float*>(A.y)[at + r] = c[r];
        else static_cast<uint16_t*>(A.y)[at + r] = (uint16_t)bf16x2(c[r], c[r]);
    }
}

// Few rows of a: a workgroup takes 16 rows of b and 16 * MT rows of a, its
// waves share out k in steps of 128 and add their results through LDS.  The
// operands go from memory to registers; each weight is read once.
constexpr int kRowsWaves = 4;

template <bool FP4B, bool FP4A, int MT>
__global__ __launch_bounds__(64 * kRowsWaves) void k_mx_matmul_rows(MatmulArgs A, int tiles_n) {
    __shared__ v4f part[kRowsWaves][MT][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int tile_m = blockIdx.x / tiles_n, tile_n = blockIdx.x - tile_m * tiles_n;
    const int n = tile_n * 16 + r;
    const bool in_n = n < A.N;
    const int64_t nr = in_n ? n : 0;
    const uint8_t* b = A.b + nr * row_bytes<FP4B>(A.K);
    const uint8_t* be = A.be + nr * (A.K / 32);
    const uint8_t *a[MT], *ae[MT];
    bool in_m[MT];
    v4f c[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int64_t m = ((int64_t)tile_m * MT + i) * 16 + r;
        in_m[i] = m < A.M;
        a[i] = A.a + (in_m[i] ? m : 0) * row_bytes<FP4A>(A.K);
        ae[i] = A.ae + (in_m[i] ? m : 0) * (A.K / 32);
        c[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    for (int k0 = wave * 128; k0 < A.K; k0 += kRowsWaves * 128) {
        const Frag<FP4B> fb = load_frag<FP4B>(b, be, in_n, k0, A.K, g);
#pragma unroll
        for (int i = 0; i < MT; i++) c[i] = mfma<FP4B, FP4A>(fb, load_frag<FP4A>(a[i], ae[i], in_m[i], k0, A.K, g), c[i]);
    }
#pragma unroll
    for (int i = 0; i < MT; i++) part[wave][i][lane] = c[i];
    __syncthreads();
    for (int i = wave; i < MT; i += kRowsWaves) {
        v4f s = part[0][i][lane];
#pragma unroll
        for (int w = 1; w < kRowsWaves; w++) s += part[w][i][lane];
        const int64_t m = ((int64_t)tile_m * MT + i) * 16 + r;
        const int at = tile_n * 16 + g * 4;
        if (m < A.M && at < A.N) store_y4(A, m, at, s);
    }
}

// Many rows: a workgroup computes a TN x TM tile of y^T from stages of the
// operands in LDS, two of them, so that a stage arrives from memory while the
// other one is computed on.  A stage holds KS steps of 128 elements (128 bytes
// of every row, or 64 of an E2M1 operand beside an E4M3 one).
//
// The loads go from memory to LDS without registers: a wave's 64 pieces of 16
// bytes land one after the other, so the order inside a stage is chosen by
// which piece each lane asks for.  Row r keeps its piece c at place c ^ s(r),
// where s counts the rows that share a place in the 256 bytes of the LDS banks:
// the 16 lanes that read the same piece of 16 rows then reach 16 different bank
// groups.  Pieces past K come from a block of zeros; rows past the end repeat
// the last row, and their results are not stored.
static __device__ __align__(16) uint32_t g_zeros[4];

template <bool FP4>
struct Stage {
    template <int KS>
    static constexpr int pitch() { return row_bytes<FP4>(128 * KS); }   // 64 or 128 bytes
    template <int KS>
    static __device__ __forceinline__ int swizzle(int row) {
        return pitch<KS>() == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
    }
    static constexpr int kElems = FP4 ? 32 : 16;   // elements of a 16-byte piece
};

// 16 bytes of each lane from memory to LDS: lane l's to byte `to` + 16 * l.  The
// compiler does not see these loads: it would wait for all of them before any
// read of LDS, the other stage's included.  lds_arrived() waits for this
// wave's own; they write no register, so nothing else depends on them.
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t to) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const uint8_t* p, uint32_t to) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void lds_arrived() { __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Workgroup b's tile.  Workgroups go to the 8 XCDs in turn, and each XCD has an
// L2 of its own: XCD x takes a run of tiles of its own, in columns of
// kTileGroup rows of tiles, so that the workgroups that run on it at one time
// share few rows of either operand.
constexpr int kXcds = 8, kTileGroup = 8;
__device__ __forceinline__ void tile_of(int b, int tiles_n, int tiles_m, int& n, int& m) {
    const int total = tiles_n * tiles_m, each = total / kXcds, more = total % kXcds;
    const int x = b % kXcds, t = x * each + (x < more ? x : more) + b / kXcds;
    const int first = t / (kTileGroup * tiles_n) * kTileGroup;
    const int rows = tiles_m - first < kTileGroup ? tiles_m - first : kTileGroup;
    const int in = t - first * tiles_n;
    m = first + in % rows;
    n = in / rows;
}

template <bool FP4B, bool FP4A>
constexpr int stage_steps() {
    return FP4B && FP4A ? 2 : 1;
}

template <bool FP4B, bool FP4A, int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM, 2) void k_mx_matmul_tile(MatmulArgs A, int tiles_n, int tiles_m) {
    constexpr int T = 64 * WN * WM, KS = stage_steps<FP4B, FP4A>(), BK = 128 * KS;
    constexpr int PB = Stage<FP4B>::template pitch<KS>(), PA = Stage<FP4A>::template pitch<KS>();
    constexpr int CB = PB / 16, CA = PA / 16;                  // 16-byte pieces of a row
    constexpr int LB = TN * CB / T, LA = TM * CA / T;          // loads of a thread
    constexpr int FN = TN / WN / 16, FM = TM / WM / 16;        // 16-row pieces of a wave
    // LDS: two stages of codes a power of two apart, then two of scale bytes, so
    // that an address goes from stage to stage by flipping one bit
    constexpr int kCodes = TN * PB + TM * PA, kScales = (TN + TM) * 4 * KS;
    constexpr int kNextCodes = 1 << (32 - __builtin_clz(kCodes - 1)), kNextScales = 1 << (32 - __builtin_clz(kScales - 1));
    constexpr int kScales0 = kNextCodes + kCodes;
    static_assert(kScales0 % (2 * kNextScales) == 0, "scale addresses flip too");
    static_assert(TN * CB % T == 0 && TM * CA % T == 0 && (T / CB) % 16 == 0 && (T / CA) % 16 == 0, "whole loads, one swizzle per lane");
    constexpr int SR = (TN + TM + T - 1) / T;                  // scale rows of a thread
    __shared__ __align__(4096) uint8_t lds[kScales0 + kNextScales + kScales];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;
    int tile_n, tile_m;
    tile_of(blockIdx.x, tiles_n, tiles_m, tile_n, tile_m);
    const int64_t n0 = (int64_t)tile_n * TN, m0 = (int64_t)tile_m * TM;
    const int pitch_b = row_bytes<FP4B>(A.K), pitch_a = row_bytes<FP4A>(A.K), blocks = A.K / 32;
    const int last_n = (int)(A.N - 1 - n0), last_m = (int)(A.M - 1 - m0);   // last rows of the tile inside

    // offsets from the tile's origin (below 2^31: K is limited by the caller)
    uint32_t off_b[LB], off_a[LA];
    const int src_b = (tid % CB) ^ Stage<FP4B>::template swizzle<KS>(tid / CB);
    const int src_a = (tid % CA) ^ Stage<FP4A>::template swizzle<KS>(tid / CA);
#pragma unroll
    for (int i = 0; i < LB; i++) {
        const int row = i * (T / CB) + tid / CB;
        off_b[i] = (uint32_t)(row < last_n ? row : last_n) * pitch_b + src_b * 16;
    }
#pragma unroll
    for (int i = 0; i < LA; i++) {
        const int row = i * (T / CA) + tid / CA;
        off_a[i] = (uint32_t)(row < last_m ? row : last_m) * pitch_a + src_a * 16;
    }
    const uint8_t* gb = A.b + n0 * pitch_b;
    const uint8_t* ga = A.a + m0 * pitch_a;
    const uint8_t* srow[SR];
#pragma unroll
    for (int i = 0; i < SR; i++) {
        const int row = i * T + tid, rm = row - TN;
        srow[i] = row < TN ? A.be + (n0 + (row < last_n ? row : last_n)) * blocks
                           : A.ae + (m0 + (rm < last_m ? rm : last_m)) * blocks;
    }

    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    uint32_t sc[SR][KS];
    // stage `step` into buffer `buf`; TAIL: the stage may pass K
    auto fetch = [&](auto tail, int step, int buf) {
        constexpr bool TAIL = decltype(tail)::value;
        const int k0 = step * BK;
        const uint8_t* pb = gb + row_bytes<FP4B>(k0);
        const uint8_t* pa = ga + row_bytes<FP4A>(k0);
        const uint32_t to = lds0 + buf * kNextCodes + wave * 1024;
        if constexpr (!TAIL) {
#pragma unroll
            for (int i = 0; i < LB; i++) load_to_lds(pb, off_b[i], to + i * T * 16);
#pragma unroll
            for (int i = 0; i < LA; i++) load_to_lds(pa, off_a[i], to + TN * PB + i * T * 16);
        } else {
            const uint8_t* z = reinterpret_cast<const uint8_t*>(g_zeros);
            const bool zb = k0 + src_b * Stage<FP4B>::kElems >= A.K, za = k0 + src_a * Stage<FP4A>::kElems >= A.K;
#pragma unroll
            for (int i = 0; i < LB; i++) load_to_lds(zb ? z : pb + off_b[i], to + i * T * 16);
#pragma unroll
            for (int i = 0; i < LA; i++) load_to_lds(za ? z : pa + off_a[i], to + TN * PB + i * T * 16);
        }
#pragma unroll
        for (int i = 0; i < SR; i++) {
            const uint8_t* p = srow[i] + k0 / 32;
#pragma unroll
            for (int j = 0; j < KS; j++) {
                if constexpr (!TAIL) {
                    __builtin_memcpy(&sc[i][j], p + 4 * j, 4);
                } else {
                    sc[i][j] = 0x7f7f7f7fu;
                    for (int x = 0; x < 4; x++)
                        if (k0 / 32 + 4 * j + x < blocks) sc[i][j] = (sc[i][j] & ~(0xffu << (8 * x))) | (uint32_t)p[4 * j + x] << (8 * x);
                }
            }
        }
    };
    auto put_scales = [&](int buf) {
#pragma unroll
        for (int i = 0; i < SR; i++)
            if ((TN + TM) % T == 0 || i * T + tid < TN + TM)
#pragma unroll
                for (int j = 0; j < KS; j++)
                    *reinterpret_cast<uint32_t*>(lds + kScales0 + buf * kNextScales + ((i * T + tid) * KS + j) * 4) = sc[i][j];
    };

    v4f c[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
        for (int j = 0; j < FM; j++) c[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int row_b = wn * FN * 16 + r, row_a = wm * FM * 16 + r;
    const int swz_b = Stage<FP4B>::template swizzle<KS>(r), swz_a = Stage<FP4A>::template swizzle<KS>(r);
    // offsets in LDS of the lane's two pieces (of an E4M3 row, or of the two steps of an E2M1
    // row) and of its scale byte in the current stage
    uint32_t b0 = row_b * PB + (g ^ swz_b) * 16, b1 = row_b * PB + ((4 + g) ^ swz_b) * 16;
    uint32_t a0 = TN * PB + row_a * PA + (g ^ swz_a) * 16, a1 = TN * PB + row_a * PA + ((4 + g) ^ swz_a) * 16;
    uint32_t sb = kScales0 + row_b * 4 * KS + g, sa = kScales0 + (TN + row_a) * 4 * KS + g;
    auto frag_b = [&](int i, int ks) {
        Frag<FP4B> f;
        f.lo = *reinterpret_cast<const v4u*>(lds + (ks ? b1 : b0) + i * 16 * PB);
        if constexpr (!FP4B) f.hi = *reinterpret_cast<const v4u*>(lds + b1 + i * 16 * PB);
        f.scale = lds[sb + i * 64 * KS + ks * 4];
        return f;
    };
    auto frag_a = [&](int i, int ks) {
        Frag<FP4A> f;
        f.lo = *reinterpret_cast<const v4u*>(lds + (ks ? a1 : a0) + i * 16 * PA);
        if constexpr (!FP4A) f.hi = *reinterpret_cast<const v4u*>(lds + a1 + i * 16 * PA);
        f.scale = lds[sa + i * 64 * KS + ks * 4];
        return f;
    };

    const int full = A.K / BK, steps = (A.K + BK - 1) / BK;   // stages, the last one may pass K
    Frag<FP4A> fa[FM];
    Frag<FP4B> fb;
    // a row of products; then(j) may load what takes the place of fa[j] from there on
    auto products = [&](int i, auto then) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < FM; j++) {
            c[i][j] = mfma<FP4B, FP4A>(fb, fa[j], c[i][j]);
            then(j);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // One stage.  Its one barrier stands where a wave has read all it needs of the
    // stage but still has a row of products to do: what follows the barrier (the
    // loads of stage s + 2 into the LDS just freed, the first reads of stage s + 1)
    // goes on beside those products.  FETCH: 0 none, 1 a full stage, 2 the last one.
    auto stage = [&](auto fetch_kind, auto last_stage, int s) {
        constexpr int FETCH = decltype(fetch_kind)::value;
        constexpr bool LAST = decltype(last_stage)::value;
        const int buf = s & 1;
#pragma unroll
        for (int i = 0; i < FN * KS - 1; i++) {
            const Frag<FP4B> next = frag_b((i + 1) % FN, (i + 1) / FN);
            products(i % FN, [&](int j) {
                if (i % FN == FN - 1) fa[j] = frag_a(j, i / FN + 1);
            });
            fb = next;
        }
        if constexpr (LAST) {
            products(FN - 1, [](int) {});
        } else {
            put_scales(buf ^ 1);
            lds_arrived();
            __syncthreads();
            if constexpr (FETCH == 1) fetch(std::false_type{}, s + 2, buf);
            if constexpr (FETCH == 2) fetch(std::true_type{}, s + 2, buf);
            b0 ^= kNextCodes, b1 ^= kNextCodes, a0 ^= kNextCodes, a1 ^= kNextCodes, sb ^= kNextScales, sa ^= kNextScales;
            const Frag<FP4B> next = frag_b(0, 0);
            products(FN - 1, [&](int j) { fa[j] = frag_a(j, 0); });
            fb = next;
        }
    };
    if (full > 0) fetch(std::false_type{}, 0, 0);
    else fetch(std::true_type{}, 0, 0);
    put_scales(0);
    lds_arrived();
    __syncthreads();
    if (full > 1) fetch(std::false_type{}, 1, 1);
    else if (steps > 1) fetch(std::true_type{}, 1, 1);
#pragma unroll
    for (int j = 0; j < FM; j++) fa[j] = frag_a(j, 0);
    fb = frag_b(0, 0);
    using std::integral_constant;
    int s = 0;
    for (; s + 2 < full; s++) stage(integral_constant<int, 1>{}, std::false_type{}, s);
    if (s + 2 < steps) stage(integral_constant<int, 2>{}, std::false_type{}, s++);
    if (s + 1 < steps) stage(integral_constant<int, 0>{}, std::false_type{}, s++);
    stage(integral_constant<int, 0>{}, std::true_type{}, s);
    // Every product is done here, by all lanes: without this the compiler moves the last
    // ones under the condition of their stores, where the lanes of rows past M, whose
    // operands the matrix instruction needs too, are switched off.
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
        for (int j = 0; j < FM; j++) __asm__ volatile("" : "+v"(c[i][j]));
#pragma unroll
    for (int j = 0; j < FM; j++) {
        const int64_t m = m0 + row_a + j * 16;
#pragma unroll
        for (int i = 0; i < FN; i++) {
            const int64_t n = n0 + wn * FN * 16 + i * 16 + g * 4;
            if (m < A.M && n < A.N) store_y4(A, m, (int)n, c[i][j]);
        }
    }
}

}  // namespace
