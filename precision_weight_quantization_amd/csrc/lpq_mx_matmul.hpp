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

}  // namespace
