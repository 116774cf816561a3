// Low-rank adapters of many requests at once, beside a shared projection: forward and
// backward.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

// Token t has adapter g (or none):  u = x[t] A_g^T,  y[t] = base[t] + s_g u B_g^T.  The tokens
// of an adapter are a run of rows of a plan (src: the token of a row), so that each tile of 16
// rows has one A and one B.  Four kinds of product:
//   shrink    U[row] = X[token] W_g^T             long contraction, `rank` results
//   expand    out[token] = in[token] + s_g U[row] W_g^T      contraction of `rank`
//   gradient  V_g^T X_g over the rows of g        contraction over tokens
//   transpose of A and B, for the backward pass's shrink and expand
// U is FP32.  It meets the BF16 matrix instruction as a sum of BF16 numbers: two for a BF16
// result (off by 2^-17 of each term, its rounding is 2^-9), three, which is all 24 bits, for
// the FP32 gradients.  Products of BF16 numbers are exact in FP32, so every sum is an FP32 one.
// Memory is the floor: x, base and y once, and the adapters' factors.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// v_mfma_f32_16x16x32_bf16: lane l holds row l % 16 and 8 consecutive elements of the
// contraction, from 8 * (l / 16) on, of both operands; result register r of lane l is row 4 *
// (l / 16) + r of the first, row l % 16 of the second.
__device__ __forceinline__ v4f mfma_bf16(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// 8 FP32 numbers as the BF16 vector nearest to them; they keep what is left.
__device__ __forceinline__ v4u take_bf16(float (&f)[8]) {
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        w[i] = bf16x2(f[2 * i], f[2 * i + 1]);
        f[2 * i] -= bf16_lo(w[i]);
        f[2 * i + 1] -= bf16_hi(w[i]);
    }
    return w;
}

// The token of a row; -1 where a plan that was not made for these tokens holds something else.
__device__ __forceinline__ int64_t token_of(const int32_t* src, int64_t row, int64_t tokens) {
    const int64_t t = src[row];
    return (uint64_t)t < (uint64_t)tokens ? t : -1;
}

struct ShrinkArgs {
    const uint16_t *x, *w;    // [tokens, K], [groups, rank, K]
    const int32_t* src;       // [capacity]
    float* u;                 // [splits, capacity, rank]: the sums of parts of k
    int64_t tokens;
    int32_t K, rank;
    int32_t splits, each;     // each: elements of a part, a multiple of 32
};

// A workgroup takes 16 * MT rows of a group, all of the rank (NT tiles) and one part of k, which
// its waves share out in steps of 32; their results are added through LDS.
constexpr int kShrinkWaves = 8;
template <int NT, int MT>
__global__ __launch_bounds__(64 * kShrinkWaves) void k_adapter_shrink(ShrinkArgs A, Routing R) {
    constexpr int W = kShrinkWaves, U = 2;   // U steps' loads go out together
    __shared__ v4f part[W][NT * MT][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const RouteMap map(R, RowTiles<16 * MT>{});
    const int v = (int)(blockIdx.x / A.splits), split = (int)(blockIdx.x % A.splits);
    if (v >= map.total) return;   // the whole workgroup
    RouteRun run;
    int within;
    const int group = map.find(R, v, run, within);
    const int first = run.first + within * 16 * MT, last = min(first + 16 * MT, run.last);
    const uint16_t *x[MT], *w[NT];
    bool in_m[MT], in_n[NT];
    v4f c[NT][MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int row = first + i * 16 + r;
        const int64_t t = row < last ? token_of(A.src, row, A.tokens) : -1;
        in_m[i] = t >= 0;
        x[i] = A.x + (in_m[i] ? t : 0) * A.K;
    }
#pragma unroll
    for (int j = 0; j < NT; j++) {
        in_n[j] = j * 16 + r < A.rank;
        w[j] = A.w + ((int64_t)group * A.rank + (in_n[j] ? j * 16 + r : 0)) * A.K;
#pragma unroll
        for (int i = 0; i < MT; i++) c[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int begin = split * A.each, end = min(begin + A.each, A.K);
    for (int k0 = begin + wave * 32 * U; k0 < end; k0 += W * 32 * U) {
        v4u fx[U][MT], fw[U][NT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k = k0 + u * 32 + 8 * g;
            const bool in = k < end;   // K % 8 == 0
#pragma unroll
            for (int i = 0; i < MT; i++) fx[u][i] = in && in_m[i] ? load<false>(reinterpret_cast<const v4u*>(x[i] + k)) : v4u{};
#pragma unroll
            for (int j = 0; j < NT; j++) fw[u][j] = in && in_n[j] ? load<false>(reinterpret_cast<const v4u*>(w[j] + k)) : v4u{};
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int i = 0; i < MT; i++) c[j][i] = mfma_bf16(fw[u][j], fx[u][i], c[j][i]);
    }
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < MT; i++) part[wave][j * MT + i][lane] = c[j][i];
    __syncthreads();
    for (int y = wave; y < NT * MT; y += W) {
        v4f s = part[0][y][lane];
#pragma unroll
        for (int i = 1; i < W; i++) s += part[i][y][lane];
        const int row = first + y % MT * 16 + r, j = y / MT * 16 + g * 4;   // 4 results: rank % 8 == 0
        if (row < last && j < A.rank)
            store<false>(reinterpret_cast<v4f*>(A.u + ((int64_t)split * R.capacity + row) * A.rank + j), s);
    }
}

struct ExpandArgs {
    const float* u;           // [splits, capacity, rank]
    const uint16_t* w;        // [groups, N, rank]
    const float* scale;       // [groups], NULL: ones
    const int32_t *rows, *src;
    const uint16_t* in;       // [tokens, N], NULL: zeros
    uint16_t* out;            // [tokens, N], may be `in`
    int64_t tokens;
    int32_t N, rank, splits;
    int32_t columns;          // of a wave, a multiple of 64
    int32_t chunks;           // parts of so many columns in N
    int32_t copy_tiles;       // of 64 tokens: the first ones look for tokens without a row
};

// A wave takes 16 rows of a group and `columns` columns, 64 at a time.  Row i of the first
// operand of its p-th instruction (of 4) is column 16 * (i / 4) + 4 * p + i % 4, so that
// the four results of a lane are 16 neighbouring columns.
constexpr int kExpandWaves = 4;
template <int STEPS>
__global__ __launch_bounds__(64 * kExpandWaves) void k_adapter_expand(ExpandArgs A, Routing R) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int chunk = (int)(blockIdx.x % A.chunks);
    int v = (int)(blockIdx.x / A.chunks) * kExpandWaves + wave;
    const int n_first = chunk * A.columns, n_last = min(n_first + A.columns, A.N);
    if (v < A.copy_tiles) {
        const int64_t t0 = (int64_t)v * 64;
        const bool none = t0 + lane < A.tokens && (uint32_t)A.rows[t0 + lane] >= (uint32_t)R.capacity;
        for (uint64_t m = __builtin_amdgcn_ballot_w64(none); m; m &= m - 1) {
            const int64_t at = (t0 + __builtin_ctzll(m)) * A.N;
            for (int n = n_first + lane * 8; n < n_last; n += 64 * 8)
                store<false>(reinterpret_cast<v4u*>(A.out + at + n), A.in ? load<false>(reinterpret_cast<const v4u*>(A.in + at + n)) : v4u{});
        }
        return;
    }
    v -= A.copy_tiles;
    const RouteMap map(R, RowTiles<16>{});
    if (v >= map.total) return;
    RouteRun run;
    int within;
    const int group = map.find(R, v, run, within);
    const int row = run.first + within * 16 + r;
    const int64_t t = row < run.last ? token_of(A.src, row, A.tokens) : -1;
    const float scale = A.scale ? A.scale[group] : 1.0f;
    v4u hi[STEPS], lo[STEPS];   // s_g u: 8 elements of the rank a step
#pragma unroll
    for (int s = 0; s < STEPS; s++) {
        float f[8];
        const int j = s * 32 + 8 * g;
        v4f a{}, b{};
        if (t >= 0 && j < A.rank) {
            for (int i = 0; i < A.splits; i++) {
                const v4f* p = reinterpret_cast<const v4f*>(A.u + ((int64_t)i * R.capacity + row) * A.rank + j);
                a += load<false>(p);
                b += load<false>(p + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = a[i] * scale, f[4 + i] = b[i] * scale;
        hi[s] = take_bf16(f);
        lo[s] = take_bf16(f);
    }
    const uint16_t* w = A.w + (int64_t)group * A.N * A.rank;
    const int64_t at = (t >= 0 ? t : 0) * A.N;
    for (int n0 = n_first; n0 < n_last; n0 += 64) {
        const int n = n0 + 16 * g;   // of this lane's results
        v4u base[2];
#pragma unroll
        for (int h = 0; h < 2; h++)   // N % 8 == 0
            base[h] = t >= 0 && A.in && n + 8 * h < n_last ? load<false>(reinterpret_cast<const v4u*>(A.in + at + n + 8 * h)) : v4u{};
        v4u fw[4][STEPS];
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const int col = n0 + 16 * (r >> 2) + 4 * p + (r & 3);
#pragma unroll
            for (int s = 0; s < STEPS; s++) {
                const int j = s * 32 + 8 * g;
                fw[p][s] = col < n_last && j < A.rank ? load<false>(reinterpret_cast<const v4u*>(w + (int64_t)col * A.rank + j)) : v4u{};
            }
        }
        v4f c[4];
#pragma unroll
        for (int p = 0; p < 4; p++) {
            c[p] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < STEPS; s++) {
                c[p] = mfma_bf16(fw[p][s], lo[s], c[p]);
                c[p] = mfma_bf16(fw[p][s], hi[s], c[p]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (t < 0 || n + 8 * h >= n_last) continue;
            const F8 f = widen8(base[h]);
            v4u o;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const v4f& d = c[2 * h + i / 2];
                o[i] = bf16x2(f.x[2 * i] + d[(i & 1) * 2], f.x[2 * i + 1] + d[(i & 1) * 2 + 1]);
            }
            store<false>(reinterpret_cast<v4u*>(A.out + at + n + 8 * h), o);
        }
    }
}

// out[g] = in[g]^T: [groups, M, N] to [groups, N, M] of 16-bit elements, 64 x 64 at a time
// through LDS.
struct AdapterTransposeArgs {
    const uint16_t* in;
    uint16_t* out;
    int32_t M, N, tiles_m, tiles_n;
};
__global__ __launch_bounds__(256) void k_adapter_transpose(AdapterTransposeArgs A) {
    __shared__ uint16_t tile[64][66];   // the odd number of words a row shifts the banks
    const int per = A.tiles_m * A.tiles_n, group = (int)blockIdx.x / per, in_group = (int)blockIdx.x - group * per;
    const int m0 = in_group / A.tiles_n * 64, n0 = in_group % A.tiles_n * 64;
    const int64_t at = (int64_t)group * A.M * A.N;
    const int x = threadIdx.x & 63;
    for (int y = threadIdx.x >> 6; y < 64; y += 4)
        if (m0 + y < A.M && n0 + x < A.N) tile[y][x] = A.in[at + (int64_t)(m0 + y) * A.N + n0 + x];
    __syncthreads();
    for (int y = threadIdx.x >> 6; y < 64; y += 4)
        if (n0 + y < A.N && m0 + x < A.M) A.out[at + (int64_t)(n0 + y) * A.M + m0 + x] = tile[x][y];
}

struct AdapterGradArgs {
    const uint16_t* x;        // [tokens, C]
    const float* v;           // [parts, capacity, rank]
    const float* scale;       // [groups], NULL: ones
    const int32_t* src;
    float* out;               // [splits, groups, rank, C] or, rank last, [splits, groups, C, rank]
    int64_t tokens;
    int32_t C, rank, parts;
    int32_t splits, tiles;    // parts of a group's rows; 128-column tiles
    int32_t rank_tiles;       // 64-element pieces of the rank
    int32_t rank_last, accumulate;
};

// out[g][j][c] = s_g * sum over the rows of g of v[row][j] x[token][c]: a workgroup takes 128
// columns, up to 64 elements of the rank and one part of the group's rows, which its waves share
// out in steps of 32; their sums are added through LDS, in wave order.  A lane loads 8 x 8
// pieces of x, 8 rows by 8 columns; column p of all pieces makes the second operand of one
// instruction: its row l % 16 is column 8 * (l % 16) + p.
constexpr int kGradWaves = 4;
template <int JT>
__global__ __launch_bounds__(64 * kGradWaves) void k_adapter_grad(AdapterGradArgs A, Routing R) {
    constexpr int W = kGradWaves;
    __shared__ v4f part[W][JT][8][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    int b = (int)blockIdx.x;
    const int tile = b % A.tiles;
    b /= A.tiles;
    const int piece = b % A.rank_tiles;
    b /= A.rank_tiles;
    const int split = b % A.splits, group = b / A.splits;
    const RouteRun run = wave_run(R, group);
    const int j0 = piece * 64, col = tile * 128 + 8 * r;
    const bool in_c = col < A.C;   // C % 8 == 0
    const float scale = A.scale ? A.scale[group] : 1.0f;
    v4f c[JT][8];
#pragma unroll
    for (int j = 0; j < JT; j++)
#pragma unroll
        for (int p = 0; p < 8; p++) c[j][p] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int row0 = run.first + (split * W + wave) * 32; row0 < run.last; row0 += A.splits * W * 32) {
        v4u x[8];
        bool in_m[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int row = row0 + 8 * g + i;
            const int64_t t = row < run.last ? token_of(A.src, row, A.tokens) : -1;
            in_m[i] = t >= 0;
            x[i] = in_m[i] && in_c ? load<false>(reinterpret_cast<const v4u*>(A.x + t * A.C + col)) : v4u{};
        }
        v4u v[JT][3];
#pragma unroll
        for (int j = 0; j < JT; j++) {
            float f[8];
            const int at = j0 + j * 16 + r;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                f[i] = 0.0f;
                if (in_m[i] && at < A.rank) {
                    for (int s = 0; s < A.parts; s++) f[i] += load<false>(A.v + ((int64_t)s * R.capacity + row0 + 8 * g + i) * A.rank + at);
                    f[i] *= scale;
                }
            }
#pragma unroll
            for (int s = 0; s < 3; s++) v[j][s] = take_bf16(f);
        }
#pragma unroll
        for (int p = 0; p < 8; p++) {
            const v4u xc = piece_column(x, p);
#pragma unroll
            for (int j = 0; j < JT; j++)
#pragma unroll
                for (int s = 2; s >= 0; s--) c[j][p] = mfma_bf16(v[j][s], xc, c[j][p]);
        }
    }
#pragma unroll
    for (int j = 0; j < JT; j++)
#pragma unroll
        for (int p = 0; p < 8; p++) part[wave][j][p][lane] = c[j][p];
    __syncthreads();
    // a wave finishes every 4th tile of the rank: for each of its lane's 4 elements 8 neighbouring columns
    float* out = A.out + ((int64_t)split * R.groups + group) * A.rank * A.C;
    for (int j = wave; j < JT; j += W) {
        v4f s[8];
#pragma unroll
        for (int p = 0; p < 8; p++) {
            s[p] = part[0][j][p][lane];
#pragma unroll
            for (int i = 1; i < W; i++) s[p] += part[i][j][p][lane];
        }
        const int at = j0 + j * 16 + 4 * g;   // 4 elements of the rank: rank % 8 == 0
        if (!in_c || at >= A.rank) continue;
        if (A.rank_last) {
#pragma unroll
            for (int p = 0; p < 8; p++) {
                v4f* to = reinterpret_cast<v4f*>(out + (int64_t)(col + p) * A.rank + at);
                store<false>(to, A.accumulate ? load<false>(to) + s[p] : s[p]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                v4f* to = reinterpret_cast<v4f*>(out + (int64_t)(at + q) * A.C + col);
                const v4f lo{s[0][q], s[1][q], s[2][q], s[3][q]}, hi{s[4][q], s[5][q], s[6][q], s[7][q]};
                store<false>(to, A.accumulate ? load<false>(to) + lo : lo);
                store<false>(to + 1, A.accumulate ? load<false>(to + 1) + hi : hi);
            }
        }
    }
}

// out (+)= the sum of `parts` arrays of n elements (n % 4 == 0), in their order.
__global__ __launch_bounds__(256) void k_adapter_sum(const float* in, float* out, int64_t n, int32_t parts, int32_t accumulate) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    v4f s = load<false>(reinterpret_cast<const v4f*>(in + i));
    for (int p = 1; p < parts; p++) s += load<false>(reinterpret_cast<const v4f*>(in + p * n + i));
    v4f* to = reinterpret_cast<v4f*>(out + i);
    store<false>(to, accumulate ? load<false>(to) + s : s);
}

}  // namespace
