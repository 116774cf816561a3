// Two-way microscaled quantization: the blocks of a matrix along its rows
// and, transposed, along its columns, from one read.
//
// Bound by memory, and in small matrices by the latency of few workgroups.  Measured,
// buffers larger than the memory-side cache (both forms / the column form alone; at the
// 5.2 TB/s of a 1 GiB copy in brackets): 8192 x 2048 in MXFP8 17.3 / 12.6 us (13.2 / 9.8),
// in MXFP4 16.5 / 12.3 (9.9 / 8.2); 1237 x 7168 in MXFP8 12.1 / 9.4 (7.0 / 5.2), in MXFP4
// 10.8 / 8.0 (5.3 / 4.3).  There 560 workgroups of 128 x 128 are two on a CU and their
// loads' latency shows; smaller tiles were not tried.  With 200 MB of buffers, part of
// them still in the cache: 13.8 us for 8192 x 2048 in MXFP8, both forms.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

// A training step multiplies a weight or an activation twice, once along its
// columns (the forward product) and once along its rows (a gradient), and a
// microscaled product needs its 1 x 32 blocks along the contraction.  So the
// column form is quantized from the BF16 values by itself (its blocks and
// scales are other ones), and is stored transposed: contraction contiguous.
//
// One workgroup takes a tile of kTrM rows by kTrN columns, four waves of 32
// rows each: a wave's lane (r, c) = (lane / 16, lane % 16) holds rows 8r to
// 8r + 7 of columns 8c to 8c + 7, an 8 x 8 piece in 32 registers.  A row block
// is a quad of lanes, as in the flat kernels; a column block is the 4 lanes of
// the same c, reduced with two lane exchanges of the 8 columns' maxima, held
// as BF16 magnitudes two to a register.  The column codes go through LDS so
// that a row of the transposed output is written 128 rows' worth at a time.
constexpr int kTrM = 128, kTrN = 128, kTrThreads = 256;

struct TransposeArgs {
    const uint16_t* w;
    uint8_t *q, *e;      // row form (NULL: not wanted)
    uint8_t *qt, *et;    // column form, transposed: [N, Mp] codes, [N, Mp / 32] scale bytes
    int64_t M, N;
    int64_t Mp;          // M rounded up to a block
    int64_t tiles_n;
    int64_t first;       // the launch's first tile
};

// Per-half maxima of two pairs of 16-bit magnitudes.
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
    const us2 r = __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b));
    return __builtin_bit_cast(uint32_t, r);
}

template <bool FP4, bool FLOOR>
__device__ __forceinline__ uint32_t mx_byte(uint32_t amax_bits) {
    if constexpr (FP4) return mx4_byte<FLOOR>(amax_bits);
    else return FLOOR ? mx_floor_scale_byte(amax_bits) : mx_scale_byte(amax_bits);
}

// 8 binary32 values -> 8 E4M3 codes, saturating under the floor rule.
template <bool FLOOR>
__device__ __forceinline__ v2u mx8_encode(F8 f, uint32_t byte) {
    if constexpr (FLOOR) {
        const float L = __uint_as_float(((byte + 8u) << 23) | 0x600000u);   // 448 * 2^(byte - 127)
#pragma unroll
        for (int k = 0; k < 8; k++) f.x[k] = __builtin_amdgcn_fmed3f(f.x[k], -L, L);
    }
    return mx_encode8(f, ue8m0_operand(byte));
}

// Column j of an 8 x 8 piece held as 8 rows of 4 words, packed as 4 words of
// two consecutive rows each.
__device__ __forceinline__ v4u piece_column(const v4u (&v)[8], int j) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t a = v[2 * i][j >> 1], b = v[2 * i + 1][j >> 1];
        // bytes of {b, a}: 0-3 are a's, 4-7 are b's
        o[i] = __builtin_amdgcn_perm(b, a, (j & 1) ? 0x07060302u : 0x05040100u);
    }
    return v4u{o[0], o[1], o[2], o[3]};
}

template <bool FP4, bool FLOOR, bool ROWS>
__global__ __launch_bounds__(kTrThreads) void k_mx_transpose(TransposeArgs A) {
    // a transposed row of the tile: 128 rows' codes; 16 more bytes shift the rows' banks
    constexpr int kRowBytes = FP4 ? kTrM / 2 : kTrM, kPitch = kRowBytes + 16;
    __shared__ __align__(16) uint8_t codes[kTrN * kPitch];
    __shared__ __align__(16) uint8_t scales[kTrN][kTrM / 32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t tile = A.first + blockIdx.x, tile_m = tile / A.tiles_n, tile_n = tile - tile_m * A.tiles_n;
    const int64_t m0 = tile_m * kTrM, n0 = tile_n * kTrN;
    const int rr = lane >> 4, cc = lane & 15;
    const int64_t row = m0 + wave * 32 + rr * 8, col = n0 + cc * 8;
    const bool in_cols = col < A.N;   // N % 32 == 0: 8 columns are all inside or all outside

    // Plain loads: the producer has just written w, and what of it is still in the
    // memory-side cache counts (non-temporal loads: 17.9 us instead of 14.0 at 8192 x 2048
    // from buffers of 100 MB together, a run before the figures above).
    v4u v[8];
#pragma unroll
    for (int p = 0; p < 8; p++) {
        const bool in = in_cols && row + p < A.M;
        v[p] = in ? load<false>(reinterpret_cast<const v4u*>(A.w + (row + p) * A.N + col)) : v4u{};
    }
    if constexpr (ROWS) {
#pragma unroll
        for (int p = 0; p < 8; p++) {
            const uint32_t byte = mx_byte<FP4, FLOOR>(quad_max(absmax8_bits(v[p])));
            if (in_cols && row + p < A.M) {
                const int64_t at = (row + p) * A.N + col;
                if constexpr (FP4) store<kNTS>(reinterpret_cast<uint32_t*>(A.q + at / 2), mx4_encode8(v[p], ue8m0_operand(byte)));
                else store<kNTS>(reinterpret_cast<v2u*>(A.q + at), mx8_encode<FLOOR>(widen8(v[p]), byte));
                if ((cc & 3) == 0) store_u8(A.e + at / 32, byte);
            }
        }
    }
    // column maxima: over the lane's 8 rows, then over the 4 lanes of the block
    uint32_t top[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        uint32_t m = v[0][k] & 0x7fff7fffu;
#pragma unroll
        for (int p = 1; p < 8; p++) m = pk_max_u16(m, v[p][k] & 0x7fff7fffu);
        m = pk_max_u16(m, (uint32_t)__shfl_xor((int)m, 16));
        top[k] = pk_max_u16(m, (uint32_t)__shfl_xor((int)m, 32));
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const uint32_t amax = (j & 1) ? top[j >> 1] & 0xffff0000u : top[j >> 1] << 16;
        const uint32_t byte = mx_byte<FP4, FLOOR>(amax);
        const v4u c = piece_column(v, j);
        uint8_t* at = codes + (cc * 8 + j) * kPitch;
        if constexpr (FP4) *reinterpret_cast<uint32_t*>(at + wave * 16 + rr * 4) = mx4_encode8(c, ue8m0_operand(byte));
        else *reinterpret_cast<v2u*>(at + wave * 32 + rr * 8) = mx8_encode<FLOOR>(widen8(c), byte);
        if (rr == 0) scales[cc * 8 + j][wave] = (uint8_t)byte;
    }
    __syncthreads();
    // the tile's transposed rows: 16-byte pieces, a row's pieces on adjacent lanes.  Rows past M
    // up to Mp are zeros of the last block; Mp % 32 == 0, so pieces are whole.
    const int64_t left = A.Mp - m0;   // rows of this tile, in elements
    constexpr int kPieces = kRowBytes / 16, kElems = FP4 ? 32 : 16;
    uint8_t* out = A.qt + (FP4 ? (n0 * A.Mp + m0) / 2 : n0 * A.Mp + m0);
    const int64_t pitch = FP4 ? A.Mp / 2 : A.Mp;
#pragma unroll
    for (int i = tid; i < kTrN * kPieces; i += kTrThreads) {
        const int n = i / kPieces, piece = i % kPieces;
        if (n0 + n < A.N && piece * kElems < left)
            store<kNTS>(reinterpret_cast<v4u*>(out + n * pitch + piece * 16), *reinterpret_cast<const v4u*>(codes + n * kPitch + piece * 16));
    }
    const int64_t blocks = A.Mp / 32;
    for (int i = tid; i < kTrN * (kTrM / 32); i += kTrThreads) {
        const int n = i / (kTrM / 32), b = i % (kTrM / 32);
        if (n0 + n < A.N && b * 32 < left) store_u8(A.et + (n0 + n) * blocks + m0 / 32 + b, scales[n][b]);
    }
}

}  // namespace
