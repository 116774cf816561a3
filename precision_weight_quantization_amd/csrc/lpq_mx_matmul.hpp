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
// Sums (measured with single products of chosen exponents).  Two E2M1 operands:
// the 32 products of a block are added exactly, then block after block to the
// accumulator, each an FP32 addition.  With an E4M3 operand: 8 consecutive products
// (aligned groups of 8 along k) are added after each has been cut towards zero to a
// multiple of 2^(X - 13), X the largest sum of two factors' exponents among the
// group's nonzero products (a subnormal code counts with the exponent of the
// smallest normal one); then group after group in FP32.  That is fewer bits than
// FP32 inside a group, and the instruction offers no other form: results on normal
// data are off by 2e-6 to 2e-5 of their root mean square, with outliers of 50 times the
// size by up to 6e-5 (lengths 128, 2560 and 16384; an FP32 sum by up to 2e-7), which
// BF16 hides, but products 2^-13 below one that cancels elsewhere are lost.  So a result with
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
    if (A.N % 4 == 0) {   // n is too: whole and aligned
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

// Few rows of a: a workgroup takes 16 * NT rows of b and 16 * MT rows of a, its
// waves share out k in steps of 128 and add their results through LDS.  The
// operands go from memory to registers; each weight is read once, and every
// workgroup reads its rows of a.  U steps' loads go out together: a wave has few
// steps, and each round trip to memory costs as much as all of them.
constexpr int kRowsWaves = 8;

template <bool FP4B, bool FP4A, int NT, int MT, int U>
__global__ __launch_bounds__(64 * kRowsWaves) void k_mx_matmul_rows(MatmulArgs A, int tiles_n, int first) {
    constexpr int W = kRowsWaves;
    __shared__ v4f part[W][NT * MT][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int tile = first + (int)blockIdx.x, tile_m = tile / tiles_n, tile_n = tile - tile_m * tiles_n;
    const uint8_t *a[MT], *ae[MT], *b[NT], *be[NT];
    bool in_m[MT], in_n[NT];
    v4f c[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
        const int64_t n = ((int64_t)tile_n * NT + j) * 16 + r;
        in_n[j] = n < A.N;
        b[j] = A.b + (in_n[j] ? n : 0) * row_bytes<FP4B>(A.K);
        be[j] = A.be + (in_n[j] ? n : 0) * (A.K / 32);
    }
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int64_t m = ((int64_t)tile_m * MT + i) * 16 + r;
        in_m[i] = m < A.M;
        a[i] = A.a + (in_m[i] ? m : 0) * row_bytes<FP4A>(A.K);
        ae[i] = A.ae + (in_m[i] ? m : 0) * (A.K / 32);
#pragma unroll
        for (int j = 0; j < NT; j++) c[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    for (int k = wave * 128; k < A.K; k += W * 128 * U) {
        Frag<FP4B> fb[U][NT];
        Frag<FP4A> fa[U][MT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k0 = k + u * W * 128;
#pragma unroll
            for (int j = 0; j < NT; j++) fb[u][j] = load_frag<FP4B>(b[j], be[j], in_n[j], k0, A.K, g);
#pragma unroll
            for (int i = 0; i < MT; i++) fa[u][i] = load_frag<FP4A>(a[i], ae[i], in_m[i], k0, A.K, g);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int i = 0; i < MT; i++) c[j][i] = mfma<FP4B, FP4A>(fb[u][j], fa[u][i], c[j][i]);
    }
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < MT; i++) part[wave][j * MT + i][lane] = c[j][i];
    __syncthreads();
    for (int x = wave; x < NT * MT; x += W) {
        v4f s = part[0][x][lane];
#pragma unroll
        for (int w = 1; w < W; w++) s += part[w][x][lane];
        const int64_t m = ((int64_t)tile_m * MT + x % MT) * 16 + r, n = ((int64_t)tile_n * NT + x / MT) * 16 + g * 4;
        if (m < A.M && n < A.N) store_y4(A, m, (int)n, s);
    }
}

// Many rows: a workgroup computes TN x TM tiles of y^T, one after the other, from
// stages of the operands in LDS, two of them, so that a stage arrives from memory
// while the other one is computed on.  A stage holds KS steps of 128 elements
// (128 bytes of every row, or 64 of an E2M1 operand beside an E4M3 one).  The
// stages of the tiles form one sequence: the next tile's first two are on their
// way before a tile's results are stored, so that the stores and the first loads
// cost no time of their own (measured with a workgroup per tile: 20 us a tile
// beside the 35 us of its products at k = 2560, MXFP8).  Measured: 8192 x 9728 x
// 2560 in MXFP8 176 us, 2.3 PFLOP/s; 8192 x 8192 x 8192 456 us, 2.4 PFLOP/s (the vendor
// library's FP8 product 360, 3.05), and 267 us in MXFP4, 4.1 PFLOP/s.
//
// The loads go from memory to LDS without registers: a wave's 64 pieces of 16
// bytes land one after the other, so the order inside a stage is chosen by
// which piece each lane asks for.  Row r keeps its piece c at place c ^ s(r),
// where s counts the rows that share a place in the 256 bytes of the LDS banks:
// the 16 lanes that read the same piece of 16 rows then reach 16 different bank
// groups (no conflicts counted).  Pieces past K load the row's last piece and are
// then overwritten with zeros.
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
// 5 wait states are what a vector memory instruction needs behind a vector
// instruction that wrote its scalar base (1 behind the write of m0); the
// compiler does not look into the block to add them.  Nor does it see the load:
// it would wait for all of them before any read of LDS, the other stage's
// included.  They write no register, so nothing
// else depends on them.  lds_arrived() waits for the wave's own.
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t to) {
    __asm__ volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(offset), "s"(uniform_ptr(base)) : "memory");
}
__device__ __forceinline__ void lds_arrived() { __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// The order of tiles.  Workgroups go to the 8 XCDs in turn, and each XCD has an
// L2 of its own: XCD x takes a run of tiles of its own, in columns of kTileGroup
// rows of tiles, so that the workgroups that run on it at one time share few
// rows of either operand.
constexpr int kXcds = 8, kTileGroup = 8;
__device__ __forceinline__ void tile_at(int t, int tiles_n, int tiles_m, int& n, int& m) {
    const int first = t / (kTileGroup * tiles_n) * kTileGroup;
    const int rows = min(tiles_m - first, kTileGroup), in = t - first * tiles_n;
    m = first + in % rows;
    n = in / rows;
}

template <bool FP4B, bool FP4A>
constexpr int stage_steps() {
    return FP4B && FP4A ? 2 : 1;
}

// f(integral_constant<int, 0>), f(integral_constant<int, 1>), ... up to N - 1.
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (N > 0) {
        static_for<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// N >= TN, M >= TM, at least two stages.
template <bool FP4B, bool FP4A, int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM, 2) void k_mx_matmul_tile(MatmulArgs A, int tiles_n, int tiles_m) {
    constexpr int T = 64 * WN * WM, KS = stage_steps<FP4B, FP4A>(), BK = 128 * KS;
    constexpr int PB = Stage<FP4B>::template pitch<KS>(), PA = Stage<FP4A>::template pitch<KS>();
    constexpr int CB = PB / 16, CA = PA / 16;                  // 16-byte pieces of a row
    constexpr int LB = TN * CB / T, LA = TM * CA / T;          // loads of a thread
    constexpr int FN = TN / WN / 16, FM = TM / WM / 16;        // 16-row pieces of a wave
    // scale rows are loaded 64 to a wave: of b by 64, of a by 64 or by wave where that is fewer
    constexpr int kRowsA = FM < 4 ? FM * 16 : 64, kChunksB = TN / 64, kChunks = kChunksB + TM / kRowsA;
    constexpr int SR = kChunks * 64 / T;                       // scale rows of a thread
    constexpr int kGroup = 4 / KS;                             // stages whose scale bytes come at once
    static_assert(TN * CB % T == 0 && TM * CA % T == 0 && (T / CB) % 16 == 0 && (T / CA) % 16 == 0, "whole loads, one swizzle per lane");
    static_assert(TN % 64 == 0 && TM % kRowsA == 0 && kChunks * 64 % T == 0 && FN % 4 == 0, "whole scale rows and result rows");
    // LDS: two stages of codes a power of two apart, so that an address goes from one to the
    // other by flipping a bit; two groups of scale bytes; 2 KB of each wave's own for results
    constexpr int kCodes = TN * PB + TM * PA, kScales = kChunks * 1024;
    constexpr int kNextCodes = 1 << (32 - __builtin_clz(kCodes - 1));
    constexpr int kScales0 = kNextCodes + kCodes, kOut = kScales0 + 2 * kScales;
    __shared__ __align__(4096) uint8_t lds[kOut + WN * WM * 2048];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;
    const int pitch_b = row_bytes<FP4B>(A.K), pitch_a = row_bytes<FP4A>(A.K), blocks = A.K / 32;
    const int full = A.K / BK, steps = (A.K + BK - 1) / BK;    // stages of a tile; the last one may pass K

    // this workgroup's tiles: every slots-th of its XCD's run
    const int total = tiles_n * tiles_m, xcd = blockIdx.x % kXcds, each = total / kXcds, more = total % kXcds;
    const int run = xcd * each + min(xcd, more), run_end = run + each + (xcd < more);
    const int slots = ((int)gridDim.x - xcd + kXcds - 1) / kXcds;

    // a lane's offsets from the first row of a load (below 2^31: K is limited by the caller)
    const int src_b = (tid % CB) ^ Stage<FP4B>::template swizzle<KS>(tid / CB);
    const int src_a = (tid % CA) ^ Stage<FP4A>::template swizzle<KS>(tid / CA);
    const uint32_t off_b = (uint32_t)(tid / CB) * pitch_b + src_b * 16, off_a = (uint32_t)(tid / CA) * pitch_a + src_a * 16;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;

    // The last tile of a row or column ends with the matrix: it repeats some of its neighbour's
    // results.
    auto origin = [&](int tile, int64_t& n0, int64_t& m0) {
        int n, m;
        tile_at(tile, tiles_n, tiles_m, n, m);
        n0 = min((int64_t)n * TN, (int64_t)A.N - TN);
        m0 = min((int64_t)m * TM, (int64_t)A.M - TM);
    };
    // the tile being loaded, its rows in memory, its next stage to load
    const int first_tile = run + blockIdx.x / kXcds;
    int load_tile = first_tile, load_step = 0;
    const uint8_t *gb = nullptr, *ga = nullptr, *gs[SR] = {};
    uint32_t off_s[SR];
#pragma unroll
    for (int i = 0; i < SR; i++)
        off_s[i] = (uint32_t)(i * T / 64 + wave < kChunksB ? lane : min(lane, kRowsA - 1)) * blocks;
    auto open_tile = [&]() {
        int64_t n0, m0;
        origin(load_tile, n0, m0);
        gb = A.b + n0 * pitch_b;
        ga = A.a + m0 * pitch_a;
#pragma unroll
        for (int i = 0; i < SR; i++) {
            const int chunk = i * T / 64 + wave;
            gs[i] = chunk < kChunksB ? A.be + (n0 + chunk * 64) * blocks : A.ae + (m0 + (chunk - kChunksB) * kRowsA) * blocks;
        }
    };
    // Scale bytes come 16 to a row, enough for kGroup stages: a row's bytes lie far from
    // the next row's, and reading 4 at each stage asks for the same lines again (measured:
    // 20 us of 233 at 8192 x 9728 x 2560).  The last group is the last 16 bytes of the row,
    // so that a group is one load (a row of fewer has one group, read byte by byte).
    auto group_start = [&](int group) { return max(min(group * 16, blocks - 16), 0); };
    v4u sc[SR];
    auto load_scales = [&](int group) {
        if (blocks >= 16) {
#pragma unroll
            for (int i = 0; i < SR; i++) __builtin_memcpy(&sc[i], gs[i] + group_start(group) + off_s[i], 16);
        } else {
#pragma unroll
            for (int i = 0; i < SR; i++) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    w[j] = 0;
#pragma unroll
                    for (int x = 0; x < 4; x++) w[j] |= (uint32_t)gs[i][off_s[i] + (4 * j + x < blocks ? 4 * j + x : 0)] << (8 * x);
                }
                sc[i] = v4u{w[0], w[1], w[2], w[3]};
            }
        }
    };
    // In LDS the bytes of 4 rows that are 16 apart lie side by side (the 64 rows of a wave's
    // load: 16 dwords for each of the 16 blocks), so that a lane reads the scales of 4 of its
    // 16-row pieces at once and each product picks its byte: a byte read for every piece took
    // 10 of 143 us (MXFP4, 8192 x 9728 x 2560).  Lane (i, r) = (lane / 16, lane % 16) holds the
    // 16 bytes of row 16 i + r: a transpose of 4 x 4 dwords over i, then of 4 x 4 bytes in place.
    auto put_scales = [&](int parity) {
#pragma unroll
        for (int i = 0; i < SR; i++) {
            const auto p02 = __builtin_amdgcn_permlane32_swap(sc[i][0], sc[i][2], false, false);
            const auto p13 = __builtin_amdgcn_permlane32_swap(sc[i][1], sc[i][3], false, false);
            const auto p01 = __builtin_amdgcn_permlane16_swap(p02[0], p13[0], false, false);
            const auto p23 = __builtin_amdgcn_permlane16_swap(p02[1], p13[1], false, false);
            uint32_t* at = reinterpret_cast<uint32_t*>(lds + kScales0 + parity * kScales + (i * T + wave * 64) * 16) + g * 64 + r;
#pragma unroll
            for (int b = 0; b < 4; b++) {
                const uint32_t pick = b | (4 + b) << 8;
                const uint32_t lo = __builtin_amdgcn_perm(p01[1], p01[0], pick), hi = __builtin_amdgcn_perm(p23[1], p23[0], pick);
                at[b * 16] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
            }
        }
    };
    auto last_piece = [&](int step, int elems) { return min(A.K - step * BK, BK) / elems - 1; };
    // the next stage of the tile being loaded, into buffer `buf`, and its scale group if it opens one
    auto load_stage = [&](int buf) {
        const int k0 = load_step * BK;
        const uint8_t* pb = gb + row_bytes<FP4B>(k0);
        const uint8_t* pa = ga + row_bytes<FP4A>(k0);
        const uint32_t to = lds0 + buf * kNextCodes + wave * 1024;
        const uint32_t ob = off_b - max(src_b - last_piece(load_step, Stage<FP4B>::kElems), 0) * 16;
        const uint32_t oa = off_a - max(src_a - last_piece(load_step, Stage<FP4A>::kElems), 0) * 16;
#pragma unroll
        for (int i = 0; i < LB; i++) load_to_lds(pb + (int64_t)i * (T / CB) * pitch_b, ob, to + i * T * 16);
#pragma unroll
        for (int i = 0; i < LA; i++) load_to_lds(pa + (int64_t)i * (T / CA) * pitch_a, oa, to + TN * PB + i * T * 16);
        if (load_step % kGroup == 0) load_scales(load_step / kGroup);
        if (++load_step == steps) {
            load_step = 0;
            load_tile += slots;
            if (load_tile < run_end) open_tile();
        }
    };
    // the pieces of stage `step` that are past K, each lane its own
    auto zero_tail = [&](int step, int buf) {
        uint8_t* at = lds + buf * kNextCodes + tid * 16;
        if (src_b > last_piece(step, Stage<FP4B>::kElems))
#pragma unroll
            for (int i = 0; i < LB; i++) *reinterpret_cast<v4u*>(at + i * T * 16) = v4u{};
        if (src_a > last_piece(step, Stage<FP4A>::kElems))
#pragma unroll
            for (int i = 0; i < LA; i++) *reinterpret_cast<v4u*>(at + TN * PB + i * T * 16) = v4u{};
    };

    // Offsets in LDS of the lane's two pieces (of an E4M3 row, or of the two steps of an E2M1
    // row) and of its scale bytes in the current stage.
    const int row_b = wn * FN * 16 + r, row_a = wm * FM * 16 + r;
    const int swz_b = Stage<FP4B>::template swizzle<KS>(r), swz_a = Stage<FP4A>::template swizzle<KS>(r);
    uint32_t b0 = row_b * PB + (g ^ swz_b) * 16, b1 = row_b * PB + ((4 + g) ^ swz_b) * 16;
    uint32_t a0 = TN * PB + row_a * PA + (g ^ swz_a) * 16, a1 = TN * PB + row_a * PA + ((4 + g) ^ swz_a) * 16;
    uint32_t sb[KS], sa[KS];
    int parity = 0;   // of the current scale group
    auto scales_of = [&](int step) {   // blocks past K take the byte of the last one (their codes are zeros)
        const int at = step * 4 * KS, start = group_start(step / kGroup), last = blocks - 1 - start;
        const uint32_t to = kScales0 + parity * kScales + r * 4;
#pragma unroll
        for (int x = 0; x < KS; x++) {
            const int y = min(at - start + x * 4 + g, last);
            sb[x] = to + wn * FN * 256 + y * 64;
            sa[x] = to + kChunksB * 1024 + wm * (TM / WM / kRowsA) * 1024 + y * 64;
        }
    };
    constexpr int SB = FN / 4, SA = (FM + 3) / 4;
    struct Scales {
        uint32_t b[SB], a[SA];
    };
    auto read_scales = [&](int ks) {
        Scales v;
#pragma unroll
        for (int i = 0; i < SB; i++) v.b[i] = *reinterpret_cast<const uint32_t*>(lds + sb[ks] + i * 1024);
#pragma unroll
        for (int j = 0; j < SA; j++) v.a[j] = *reinterpret_cast<const uint32_t*>(lds + sa[ks] + j * 1024);
        return v;
    };
    auto frag_b = [&](int i, int ks) {
        Frag<FP4B> f;
        f.lo = *reinterpret_cast<const v4u*>(lds + (ks ? b1 : b0) + i * 16 * PB);
        if constexpr (!FP4B) f.hi = *reinterpret_cast<const v4u*>(lds + b1 + i * 16 * PB);
        return f;
    };
    auto frag_a = [&](int i, int ks) {
        Frag<FP4A> f;
        f.lo = *reinterpret_cast<const v4u*>(lds + (ks ? a1 : a0) + i * 16 * PA);
        if constexpr (!FP4A) f.hi = *reinterpret_cast<const v4u*>(lds + a1 + i * 16 * PA);
        return f;
    };

    v4f c[FN][FM];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < FN; i++)
#pragma unroll
            for (int j = 0; j < FM; j++) c[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    };
    // Keeps the products in front of this point.  They have no side effects, so the compiler
    // may otherwise move them to where their results are next used: past a barrier, or under
    // a condition, where lanes that hold operands of theirs are switched off.
    auto pin = [&]() {
#pragma unroll
        for (int i = 0; i < FN; i++)
#pragma unroll
            for (int j = 0; j < FM; j++) __asm__ volatile("" : "+v"(c[i][j]));
    };
    Frag<FP4A> fa[FM];
    // Rows of b are read kAhead rows before their products: an E2M1 row's products take half as
    // long as an E4M3 row's, and the read no less.
    constexpr int kAhead = FP4B && FP4A ? 2 : 1;
    Frag<FP4B> fb[kAhead];
    Scales sv;
    // a row of products; then(j) may load what takes the place of fa[j] from there on
    auto products = [&](auto row, auto then) {
        constexpr int i = decltype(row)::value;
        __builtin_amdgcn_sched_barrier(0);
        static_for<FM>([&](auto col) {
            constexpr int j = decltype(col)::value;
            c[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag_regs(fb[0]), frag_regs(fa[j]), c[i][j], FP4B ? 4 : 0,
                                                                       FP4A ? 4 : 0, i % 4, (int)sv.b[i / 4], j % 4, (int)sv.a[j / 4]);
            then(j);
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    open_tile();
    load_stage(0);
    put_scales(0);
    lds_arrived();
    __syncthreads();
    load_stage(1);
    scales_of(0);
#pragma unroll
    for (int j = 0; j < FM; j++) fa[j] = frag_a(j, 0);
    auto first_rows = [&]() {
#pragma unroll
        for (int i = 0; i < kAhead; i++) fb[i] = frag_b(i, 0);
    };
    first_rows();
    sv = read_scales(0);

    int buf = 0;
    for (int tile = first_tile; tile < run_end; tile += slots) {
        clear();
        for (int s = 0; s < steps; s++) {
            static_for<FN * KS - 1>([&](auto at) {
                constexpr int x = decltype(at)::value, i = x % FN, ks = x / FN;
                Frag<FP4B> next = fb[kAhead - 1];
                if constexpr (x + kAhead < FN * KS) next = frag_b((x + kAhead) % FN, (x + kAhead) / FN);
                if constexpr (i == FN - 1) {   // of the stage's first step, with the reads of its second
                    const Scales next_sv = read_scales(ks + 1);
                    products(std::integral_constant<int, i>{}, [&](int j) { fa[j] = frag_a(j, ks + 1); });
                    sv = next_sv;
                } else {
                    products(std::integral_constant<int, i>{}, [](int) {});
                }
#pragma unroll
                for (int k = 0; k + 1 < kAhead; k++) fb[k] = fb[k + 1];
                fb[kAhead - 1] = next;
            });
            // The stage's one barrier, where a wave has read all it needs of the stage but
            // still has a row of products to do: what follows (the loads of the stage after
            // the next into the LDS just freed, the first reads of the next) goes on beside
            // those products.
            pin();
            const int next_step = s + 1 == steps ? 0 : s + 1;
            if (next_step % kGroup == 0) put_scales(parity ^ 1);
            lds_arrived();
            if (next_step == full) zero_tail(next_step, buf ^ 1);
            __syncthreads();
            if (load_tile < run_end) load_stage(buf);   // of this tile or of the next
            buf ^= 1;
            parity ^= next_step % kGroup == 0;
            b0 ^= kNextCodes, b1 ^= kNextCodes, a0 ^= kNextCodes, a1 ^= kNextCodes;
            scales_of(next_step);
            Frag<FP4B> next[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; i++) next[i] = frag_b(i, 0);
            const Scales next_sv = read_scales(0);
            products(std::integral_constant<int, FN - 1>{}, [&](int j) { fa[j] = frag_a(j, 0); });
            sv = next_sv;
#pragma unroll
            for (int i = 0; i < kAhead; i++) fb[i] = next[i];
            pin();
        }
        int64_t n0, m0;
        origin(tile, n0, m0);
        n0 += wn * FN * 16, m0 += wm * FM * 16;
        int N = A.N;   // opaque here: else the offsets of every store are formed before the first tile and kept
        __asm__ volatile("" : "+s"(N));
        // Rows by way of LDS, 16 rows of 128 bytes at a time, so that 128 bytes of a row leave
        // in one piece: stored from the accumulators each instruction would write 32 bytes of
        // 16 rows (measured: 17 us of 233 at 8192 x 9728 x 2560).  Swizzled as a stage's rows
        // are.  Non-temporal: 9 us of 207 there.
        auto store_rows = [&](auto f32) {
            constexpr bool F32 = decltype(f32)::value;
            constexpr int kSize = F32 ? 4 : 2, kFrags = F32 ? 2 : 4;   // 16-column results in 128 bytes
            uint8_t* mine = lds + kOut + wave * 2048;
            uint8_t* y = static_cast<uint8_t*>(A.y) + (m0 * N + n0) * kSize;   // uniform
            const uint32_t off = (uint32_t)(lane >> 3) * N * kSize + (lane & 7) * 16;
#pragma unroll
            for (int j = 0; j < FM; j++) {
#pragma unroll
                for (int h = 0; h < FN; h += kFrags) {
#pragma unroll
                    for (int i = 0; i < kFrags; i++) {
                        const v4f v = c[h + i][j];
                        if constexpr (F32)
                            *reinterpret_cast<v4f*>(mine + r * 128 + ((i * 4 + g) ^ ((r >> 1) & 7)) * 16) = v;
                        else
                            *reinterpret_cast<v2u*>(mine + r * 128 + ((i * 2 + (g >> 1)) ^ ((r >> 1) & 7)) * 16 + (g & 1) * 8) =
                                v2u{bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                    for (int x = 0; x < 16; x += 8) {
                        const int row = x + (lane >> 3);
                        const v4u v = *reinterpret_cast<const v4u*>(mine + row * 128 + ((lane & 7) ^ ((row >> 1) & 7)) * 16);
                        store<true>(reinterpret_cast<v4u*>(y + ((int64_t)(j * 16 + x) * N + h * 16) * kSize + off), v);
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                }
            }
        };
        if (A.f32 ? N % 4 == 0 : N % 8 == 0) {
            if (A.f32) store_rows(std::true_type{});
            else store_rows(std::false_type{});
        } else {
            uint8_t* y = static_cast<uint8_t*>(A.y) + (m0 * N + n0) * (A.f32 ? 4 : 2);
#pragma unroll
            for (int j = 0; j < FM; j++)
#pragma unroll
                for (int i = 0; i < FN; i++)
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        const uint32_t at = (uint32_t)(j * 16 + r) * N + i * 16 + g * 4 + x;
                        if (A.f32) store<false>(reinterpret_cast<float*>(y) + at, c[i][j][x]);
                        else store<false>(reinterpret_cast<uint16_t*>(y) + at, (uint16_t)bf16x2(c[i][j][x], 0.0f));
                    }
        }
    }
}

}  // namespace
