// Host side of the routed layers: argument checks and launches.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

struct Range {
    const void* p;
    int64_t n;   // bytes; an absent array has none
};
inline Range range(const void* p, int64_t n) { return {p, p ? n : 0}; }

// An output that shares a byte with an input or another output.
template <int O, int I>
bool any_overlap(const Range (&out)[O], const Range (&in)[I]) {
    for (int i = 0; i < O; i++) {
        for (const Range& r : in)
            if (overlap(out[i].p, out[i].n, r.p, r.n)) return true;
        for (int j = 0; j < i; j++)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    }
    return false;
}

// Rows of a routed matrix are counted in 32 bits, pairs too.
constexpr int64_t kRouteMaxRows = int64_t(1) << 30;

int64_t route_capacity(int64_t pairs, int32_t groups, int32_t align) {
    if (pairs <= 0 || pairs > kRouteMaxRows || groups <= 0 || groups > kRouteMaxGroups || align <= 0 || align > 1024) return 0;
    const int64_t most = pairs + (pairs < groups ? pairs : groups) * (int64_t)(align - 1), c = ceil_div(most, align) * align;
    return c <= kRouteMaxRows ? c : 0;
}

// Workgroups of a plan: runs of whole kPlanThreads pairs.
int64_t plan_runs(int64_t pairs) {
    if (pairs <= kPlanOne) return 1;
    const int64_t run = ceil_div(ceil_div(pairs, kPlanThreads), kPlanMaxRuns) * kPlanThreads;
    return ceil_div(pairs, run);
}

template <typename Id>
lpq_status route_plan(PlanArgs A, hipStream_t s) {
    const int64_t runs = plan_runs(A.pairs);
    A.run = ceil_div(ceil_div(A.pairs, kPlanThreads), runs) * kPlanThreads;
    if (runs == 1) A.counts = nullptr;
    else {
        hipLaunchKernelGGL(k_route_count<Id>, dim3((unsigned)runs), dim3(kPlanThreads), 0, s, A);
        const lpq_status st = launched();
        if (st != LPQ_OK) return st;
    }
    hipLaunchKernelGGL(k_route_place<Id>, dim3((unsigned)runs), dim3(kPlanThreads), 0, s, A);
    return launched();
}

// Shape of tokens with k rows each in a routed matrix of `capacity` rows, N elements a row.
lpq_status route_shape(int64_t tokens, int64_t k, int64_t capacity, int64_t N) {
    if (tokens <= 0 || k <= 0 || capacity <= 0 || N <= 0 || N % 32) return LPQ_ERR_SHAPE;
    if (N > kRouteMaxRows || capacity > kRouteMaxRows || tokens > kRouteMaxRows / k) return LPQ_ERR_SHAPE;
    if (tokens > (int64_t(1) << 40) / N || capacity > (int64_t(1) << 40) / N) return LPQ_ERR_SHAPE;
    return LPQ_OK;
}

template <int FORMAT>
lpq_status route_gather(const uint16_t* x, int64_t tokens, int64_t N, const int32_t* rows, int64_t k, const int32_t* src,
                        int64_t capacity, void* q, uint8_t* e, void* stream) {
    const lpq_status st = route_shape(tokens, k, capacity, N);
    if (st != LPQ_OK) return st;
    const int64_t pad = ceil_div(capacity, kPadRows), blocks = pad + ceil_div(tokens * (N / 8), kRouteThreads);
    if (blocks > max_groups(kRouteThreads)) return LPQ_ERR_SHAPE;
    if (!x || !rows || !src || !q || (FORMAT != ROW_BF16 && !e)) return LPQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(rows, 4) || !aligned(src, 4)) return LPQ_ERR_ALIGN;
    const int64_t size = FORMAT == ROW_BF16 ? 2 * capacity * N : FORMAT == ROW_FP8 ? capacity * N : capacity * N / 2;
    if (any_overlap({range(q, size), range(e, capacity * N / 32)},
                    {range(x, 2 * tokens * N), range(rows, 4 * tokens * k), range(src, 4 * capacity)}))
        return LPQ_ERR_ARG;
    const GatherArgs A{x, rows, src, static_cast<uint8_t*>(q), e, tokens, capacity, (int32_t)k, (int32_t)N, (int32_t)pad};
    hipLaunchKernelGGL(k_route_gather<FORMAT>, dim3((unsigned)blocks), dim3(kRouteThreads), 0, (hipStream_t)stream, A);
    return launched();
}

// The checks of a routed product: a [M, K], b [rows_b, K], y of ny elements, and the plan's offsets.
struct RoutedProduct {
    const uint8_t *a, *ae, *b, *be;
    int a_format, b_format;
    const int32_t* offsets;
    int32_t groups;
    int64_t M, rows_b, N, K, ny;
    void* y;
    int y_type;
};
lpq_status check_routed(const RoutedProduct& P) {
    if (!P.a || !P.ae || !P.b || !P.be || !P.y || !P.offsets) return LPQ_ERR_NULL;
    const bool a4 = P.a_format == LPQ_MXFP4, b4 = P.b_format == LPQ_MXFP4;
    if ((!a4 && P.a_format != LPQ_MXFP8) || (!b4 && P.b_format != LPQ_MXFP8)) return LPQ_ERR_ARG;
    if (P.y_type != LPQ_BF16 && !(P.y_type == LPQ_F32 && a4 && b4)) return LPQ_ERR_ARG;
    if (!aligned(P.a, 16) || !aligned(P.b, 16) || !aligned(P.y, 16) || !aligned(P.offsets, 4)) return LPQ_ERR_ALIGN;
    if (any_overlap({range(P.y, P.ny * (P.y_type == LPQ_F32 ? 4 : 2))},
                    {range(P.a, P.M * P.K / (a4 ? 2 : 1)), range(P.ae, P.M * P.K / 32), range(P.b, P.rows_b * P.K / (b4 ? 2 : 1)),
                     range(P.be, P.rows_b * P.K / 32), range(P.offsets, 4 * (P.groups + 1))}))
        return LPQ_ERR_ARG;
    return LPQ_OK;
}

template <bool FP4A, bool FP4B, TileMode MODE>
struct RoutedLaunch {
    MatmulArgs A;
    Routing R;
    hipStream_t s;

    // Row tiles of 16 * MT rows, in all groups together, at most.
    int64_t row_tiles(int64_t tm) const {
        const int64_t most = R.capacity < R.groups ? R.capacity : R.groups;
        return R.capacity / tm + most;
    }
    template <int NT, int MT, int U, int W>
    lpq_status rows() const {
        const int64_t tiles_n = ceil_div(A.N, 16 * NT * (kRowsWaves / W)), tiles_m = MODE == ROUTED_K ? ceil_div(A.M, 16 * MT) : 1;
        const int64_t tiles = MODE == ROUTED_K ? tiles_n * tiles_m * R.groups : tiles_n * row_tiles(16 * MT);
        const int64_t most = max_groups(64 * kRowsWaves);
        if (tiles > 0x7fffffffLL) return LPQ_ERR_SHAPE;   // tile indexes are 32-bit
        for (int64_t first = 0; first < tiles; first += most) {
            hipLaunchKernelGGL((k_mx_matmul_routed_rows<FP4B, FP4A, NT, MT, U, W, MODE>),
                               dim3((unsigned)(tiles - first < most ? tiles - first : most)), dim3(64 * kRowsWaves), 0, s, A,
                               (int)tiles_n, (int)tiles_m, R, (int)first);
            const lpq_status st = launched();
            if (st != LPQ_OK) return st;
        }
        return LPQ_OK;
    }
    template <int TN, int TM, int WN, int WM>
    lpq_status tile() const {
        const int64_t nt = ceil_div(A.N, TN), mt = MODE == ROUTED_K ? ceil_div(A.M, TM) : row_tiles(TM);
        const int64_t tiles = MODE == ROUTED_K ? nt * mt * R.groups : nt * mt;
        if (tiles > 0x7fffffffLL) return LPQ_ERR_SHAPE;
        const int64_t most = kComputeUnits * (TN == 256 ? 1 : 2);
        hipLaunchKernelGGL((k_mx_matmul_routed_tile<FP4B, FP4A, TN, TM, WN, WM, MODE>), dim3((unsigned)(tiles < most ? tiles : most)),
                           dim3(64 * WN * WM), 0, s, A, (int)nt, (int)mt, R);
        return launched();
    }
};

// Which kernel, by the rows that a group has on average (the counts themselves are on the device).  All sides
// were timed with rows drawn for 128 groups of N = 1536, k = 2048 or N = 2048, k = 768 unless said, some experts liked
// more than others; us, MXFP8 unless said:
//  * Tiles by way of LDS from 6 rows on: 4 rows 69 in tiles of 64 rows and 73 by rows, but 27 and 25 with MXFP4
//    weights (k = 768), 12 and 11 for 60 groups of 1024 x 1056; 6 rows 71 and 84; 8 rows 74 and 91. A tile's stages take
//    as long as its weights, whatever its rows.
//  * 128 x 64 tiles below 72 rows: 8 rows 74, with 128 x 128 81; 50 rows 108 and 107; 75 rows 120 and 112, evenly
//    routed 139 and 101.  So the two are even from 50 rows on in MXFP8; the border is above 70 for products of two
//    MXFP4 operands with few stages, 70 rows of 60 groups of 1024 x 1056 20 and 24.
//  * 256 x 256 from 144 rows on (evenly routed): 75 rows 130 against 101 with 128 x 128, 125 rows 108 and 102 (MXFP4
//    weights), 150 rows 123 and 149, 200 rows 134 and 157; 250 rows 186 and 178, where most groups just need a second
//    tile.  256 x 128: 163 at 150 rows, 323 instead of 276 for the workload of 512.
//  * Rows: 16 rows a tile up to 16 on average, 32 above.  Columns of a wave: as many as leave a few waves for each
//    SIMD (1 token of 8 experts, N = 2048, k = 768, MXFP4 weights: 4.7 with 16 columns, 5.6 with 32, 7.8 with 64; 24
//    tokens 31, 27 and 25; where k is long the loads in flight count: 4 tokens, N = 4096, k = 7168 161 with 32, 186
//    with 64).  Waves that share out k: of 3 steps at least (24 tokens, N = 2048, k = 768: 37 with 8, 31 with 2, 27 with
//    1; 4 tokens, N = 4096, k = 7168: 167 with 8, 179 with 4).
// The rule looks at capacity, which counts pairs without a row and padding too, and not at the number of tiles: 2
// groups of 300 rows, N = 512, k = 2048 make 8 tiles of 256 x 256 and take 29 us, 5 of 190 rows, N = 930 20 tiles and 41.
template <bool FP4A, bool FP4B>
lpq_status mx_matmul_routed(const MatmulArgs& A, const Routing& R, hipStream_t s) {
    const RoutedLaunch<FP4A, FP4B, ROUTED_ROWS> L{A, R, s};
    const int64_t average = R.capacity / R.groups;
    const bool limits = A.K > 128 * stage_steps<FP4B, FP4A>() && A.K <= (1 << 22) && A.N <= (1 << 22);
    if (limits && average >= 6 && A.N >= 128 && R.capacity >= 64) {
        if (average >= 144 && A.N >= 256 && R.capacity >= 256) return L.template tile<256, 256, 2, 4>();
        if (average >= 72 && R.capacity >= 128) return L.template tile<128, 128, 2, 2>();
        return L.template tile<128, 64, 2, 2>();
    }
    const int64_t steps = ceil_div(A.K, 128), tiles = L.row_tiles(16) * ceil_div(A.N, 64);
    auto by_share = [&](auto nt, auto mt, auto u) {
        constexpr int NT = decltype(nt)::value, MT = decltype(mt)::value, U = decltype(u)::value;
        if (steps >= 24) return L.template rows<NT, MT, U, 8>();
        if (steps >= 12) return L.template rows<NT, MT, U, 4>();
        return steps >= 6 ? L.template rows<NT, MT, U, 2>() : L.template rows<NT, MT, U, 1>();
    };
    if (average > 16) return by_share(Int<4>{}, Int<2>{}, Int<1>{});
    if (tiles > 2048 && steps < 24) return by_share(Int<4>{}, Int<1>{}, Int<1>{});
    return tiles > 512 ? by_share(Int<2>{}, Int<1>{}, Int<3>{}) : by_share(Int<1>{}, Int<1>{}, Int<3>{});
}

// Which tile, by rounds of the card as for the dense products: one of 256 x 256 counts 2, of 128 x 128 0.95
// alone, 1.1 with two on each CU and 1.4 where many rounds keep memory busy.  us, 256 x 256 and 128 x 128: 128 groups
// of 256 rows, 1536 x 2048 in MXFP8 271 and 376; of 32 rows 199 and 260; 96 groups of 32 rows, 520 x 776 in MXFP4 with an
// FP32 result 60 and 54; 60 of 512 rows, 1024 x 1024 54 and 53; 8 of 4096 rows, 1024 x 1024 in MXFP8 58 and 42.  Fewer than
// 64 tiles of long contractions leave the card idle, and nothing shares out k: 32 x 32 by 8 waves then
// (3 groups of 6269 rows, 288 x 344, MXFP4 and MXFP8: 23 us, in tiles 88).
template <bool FP4A, bool FP4B>
lpq_status mx_matmul_routed_dw(const MatmulArgs& A, const Routing& R, hipStream_t s) {
    const RoutedLaunch<FP4A, FP4B, ROUTED_K> L{A, R, s};
    const bool limits = A.K <= (1 << 22) && A.N <= (1 << 22);
    const int64_t n128 = ceil_div(A.N, 128) * ceil_div(A.M, 128) * R.groups, steps = A.K / R.groups / 128;
    if (limits && A.M >= 128 && A.N >= 128 && (n128 >= 64 || steps < 8)) {
        const int64_t n256 = ceil_div(A.N, 256) * ceil_div(A.M, 256) * R.groups;
        const double c128 = n128 <= 256 ? 0.95 : ceil_div(n128, 512) * (n128 <= 2048 ? 1.1 : 1.4);
        if (A.M >= 256 && A.N >= 256 && 2.0 * ceil_div(n256, 256) < c128) return L.template tile<256, 256, 2, 4>();
        return L.template tile<128, 128, 2, 2>();
    }
    if (steps >= 16) return L.template rows<2, 2, 2, 8>();
    return steps >= 8 ? L.template rows<2, 2, 2, 4>() : L.template rows<2, 2, 2, 2>();
}

// Adapters of one shape: x [tokens, K], y [tokens, N], factors of `rank`, rows in a plan.
struct Adapters {
    int64_t tokens, capacity;
    int32_t groups, rank;
    int64_t N, K;
};
// The launches by rows or factors of these limits stay below max_groups(): shrinks 2^21 of 512 threads, gradients
// 2^23 and planes 2^22 of 256.  Those by rows and columns together are counted by adapters_forward_shape() and
// adapters_backward_shape(), so that nothing is refused once a part is enqueued.
lpq_status adapters_shape(const Adapters& P) {
    const int64_t most = int64_t(1) << 35;
    if (P.groups <= 0 || P.groups > kRouteMaxGroups || P.rank <= 0 || P.rank > 128 || P.rank % 8) return LPQ_ERR_SHAPE;
    if (P.N <= 0 || P.K <= 0 || P.N % 8 || P.K % 8 || P.tokens <= 0 || P.capacity <= 0) return LPQ_ERR_SHAPE;
    if (P.N > (1 << 18) || P.K > (1 << 18) || P.tokens > (1 << 24) || P.capacity > (1 << 24)) return LPQ_ERR_SHAPE;
    return P.tokens > most / P.N || P.tokens > most / P.K ? LPQ_ERR_SHAPE : LPQ_OK;
}
// Tiles of 16 * mt rows: at most, and about.
int64_t adapter_tiles(const Adapters& P, int mt) { return P.capacity / (16 * mt) + (P.capacity < P.groups ? P.capacity : P.groups); }

// The shrink's rows a workgroup: 32 where the accumulators of the rank's tiles leave room.
int shrink_mt(const Adapters& P) { return P.rank <= 64 ? 2 : 1; }
// Parts of its contraction: enough workgroups for the card, of 512 elements at least.
int32_t shrink_splits(const Adapters& P, int64_t k) {
    const int64_t groups = P.capacity < P.groups ? P.capacity : P.groups, tiles = ceil_div(P.capacity, 16 * shrink_mt(P));
    int64_t s = kComputeUnits / (tiles > groups ? tiles : groups);
    if (s > k / 512) s = k / 512;
    return (int32_t)(s < 1 ? 1 : s > 16 ? 16 : s);
}
int64_t shrink_bytes(const Adapters& P, int64_t k) { return 4 * (int64_t)shrink_splits(P, k) * P.capacity * P.rank; }

struct Factor {
    const uint16_t *x, *w;
    float* u;
    int64_t k;   // 0: none
};
lpq_status adapter_shrink(const Adapters& P, const Routing& R, const Factor& one, const Factor& two, const int32_t* src, hipStream_t s) {
    const int mt = shrink_mt(P), nt = (P.rank + 15) / 16;
    const int64_t tiles = adapter_tiles(P, mt);
    ShrinkPair A{{}, src, P.tokens, P.rank};
    int64_t blocks = 0;
    for (int i = 0; i < 2; i++) {
        const Factor& f = i ? two : one;
        if (!f.k) continue;
        const int32_t splits = shrink_splits(P, f.k);
        A.a[i] = ShrinkArgs{f.x, f.w, f.u, (int32_t)f.k, splits, (int32_t)(ceil_div(ceil_div(f.k, 32), splits) * 32), (int32_t)(tiles * splits)};
        blocks += tiles * splits;
    }
    const dim3 grid((unsigned)blocks), block(64 * kShrinkWaves);
    if (nt == 1) hipLaunchKernelGGL((k_adapter_shrink<1, 2, 4>), grid, block, 0, s, A, R);
    else if (nt == 2) hipLaunchKernelGGL((k_adapter_shrink<2, 2, 4>), grid, block, 0, s, A, R);
    else if (nt <= 4) hipLaunchKernelGGL((k_adapter_shrink<4, 2, 4>), grid, block, 0, s, A, R);
    else hipLaunchKernelGGL((k_adapter_shrink<8, 1, 2>), grid, block, 0, s, A, R);
    return launched();
}

// The expand's kernel: tiles of 64 rows where a group has as many on average; else 16 rows and 256
// columns a wave, fewer columns where that leaves the card idle.
struct ExpandShape {
    bool tile;
    int64_t columns;    // of a workgroup
    int64_t copy_tiles, chunks, blocks;
};
ExpandShape expand_shape(const Adapters& P, int64_t n, int64_t copies) {
    ExpandShape e{P.capacity / P.groups >= 64, kTileColumns, 0, 0, 0};
    if (e.tile) {
        e.copy_tiles = ceil_div(copies, 64 * kExpandWaves);
        e.chunks = ceil_div(n, e.columns);
        e.blocks = (e.copy_tiles + adapter_tiles(P, 4)) * e.chunks;
        return e;
    }
    e.copy_tiles = ceil_div(copies, 64);
    const int64_t rows = ceil_div(e.copy_tiles + adapter_tiles(P, 1), kExpandWaves);
    e.columns = 256;
    while (e.columns > 64 && rows * ceil_div(n, e.columns) < 4 * kComputeUnits) e.columns /= 2;
    e.chunks = ceil_div(n, e.columns);
    e.blocks = rows * e.chunks;
    return e;
}
template <int STEPS>
lpq_status adapter_expand(ExpandArgs A, const Adapters& P, const Routing& R, hipStream_t s) {
    const ExpandShape e = expand_shape(P, A.N, A.in == A.out ? 0 : P.tokens);
    A.copy_tiles = (int32_t)e.copy_tiles;
    A.chunks = (int32_t)e.chunks;
    const dim3 grid((unsigned)e.blocks), block(64 * kExpandWaves);
    if (e.tile) hipLaunchKernelGGL(k_adapter_expand_tile<STEPS>, grid, block, 0, s, A, R);
    else if (e.columns == 256) hipLaunchKernelGGL((k_adapter_expand<STEPS, 4>), grid, block, 0, s, A, R);
    else if (e.columns == 128) hipLaunchKernelGGL((k_adapter_expand<STEPS, 2>), grid, block, 0, s, A, R);
    else hipLaunchKernelGGL((k_adapter_expand<STEPS, 1>), grid, block, 0, s, A, R);
    return launched();
}
lpq_status adapter_expand(const Adapters& P, const Routing& R, const float* u, int32_t splits, const uint16_t* w, int64_t n,
                          const float* scale, const int32_t* rows, const int32_t* src, const uint16_t* in, uint16_t* out, hipStream_t s) {
    const ExpandArgs A{u, w, scale, rows, src, in, out, P.tokens, (int32_t)n, P.rank, splits, 0, 0};
    if (P.rank <= 32) return adapter_expand<1>(A, P, R, s);
    return P.rank <= 64 ? adapter_expand<2>(A, P, R, s) : adapter_expand<4>(A, P, R, s);
}

// Parts of a group's rows in its gradients: enough workgroups for the card, of 128 rows at least.
int32_t grad_splits(const Adapters& P, int64_t c) {
    const int64_t wgs = ceil_div(c, 128) * ceil_div(P.rank, 64) * P.groups, most = ceil_div(P.capacity, 128);
    int64_t s = 2 * kComputeUnits / wgs;
    if (s > most) s = most;
    return (int32_t)(s < 1 ? 1 : s > 32 ? 32 : s);
}
int64_t grad_bytes(const Adapters& P, int64_t c) {
    const int32_t s = grad_splits(P, c);
    return s == 1 ? 0 : 4 * (int64_t)s * P.groups * P.rank * c;
}
int64_t planes_pitch(const Adapters& P) { return ceil_div(P.capacity + 32, 64) * 64; }   // a step may pass the rows by 31
int64_t planes_bytes(const Adapters& P) { return 3 * 2 * P.rank * planes_pitch(P); }

struct Gradient {
    const uint16_t* x;
    int64_t c;
    const uint16_t* planes;
    float *partial, *out;
    int rank_last;
};
lpq_status adapter_grad(const Adapters& P, const Routing& R, const Gradient (&g)[2], const float* scale, const int32_t* src,
                        int accumulate, hipStream_t s) {
    const int32_t pieces = (int32_t)ceil_div(P.rank, 64);
    AdapterGradPair A{{}, scale, src, P.tokens, P.rank, (int32_t)planes_pitch(P), pieces};
    AdapterSumArgs sum{};
    int64_t blocks = 0, sums = 0;
    for (int i = 0; i < 2; i++) {
        const int32_t splits = grad_splits(P, g[i].c), tiles = (int32_t)ceil_div(g[i].c, 128);
        const int64_t here = (int64_t)tiles * pieces * P.groups * splits, n = (int64_t)P.groups * P.rank * g[i].c;
        A.a[i] = AdapterGradArgs{g[i].x, g[i].planes, splits == 1 ? g[i].out : g[i].partial, (int32_t)g[i].c, splits, tiles, g[i].rank_last,
                                 splits == 1 ? accumulate : 0, (int32_t)here};
        blocks += here;
        sum.in[i] = g[i].partial;
        sum.out[i] = g[i].out;
        sum.n[i] = splits == 1 ? 0 : n;
        sum.parts[i] = splits;
        if (splits > 1) sums += ceil_div(n, 1024);
        if (i == 0) sum.blocks = (int32_t)sums;
    }
    sum.accumulate = accumulate;
    const dim3 grid((unsigned)blocks), block(64 * kGradWaves);
    if (P.rank <= 16) hipLaunchKernelGGL(k_adapter_grad<1>, grid, block, 0, s, A, R);
    else if (P.rank <= 32) hipLaunchKernelGGL(k_adapter_grad<2>, grid, block, 0, s, A, R);
    else hipLaunchKernelGGL(k_adapter_grad<4>, grid, block, 0, s, A, R);
    const lpq_status st = launched();
    if (st != LPQ_OK || sums == 0) return st;
    hipLaunchKernelGGL(k_adapter_sum, dim3((unsigned)sums), dim3(256), 0, s, sum);
    return launched();
}

// A^T and B^T.
AdapterTransposePair transpose_pair(const Adapters& P, const uint16_t* A, uint16_t* At, const uint16_t* B, uint16_t* Bt) {
    auto one = [&](const uint16_t* in, uint16_t* out, int64_t m, int64_t n) {
        const int32_t tm = (int32_t)ceil_div(m, 64), tn = (int32_t)ceil_div(n, 64);
        return AdapterTransposeArgs{in, out, (int32_t)m, (int32_t)n, tm, tn, P.groups * tm * tn};
    };
    return {{one(A, At, P.rank, P.K), one(B, Bt, P.N, P.rank)}};
}
lpq_status adapter_transpose(const AdapterTransposePair& T, hipStream_t s) {
    hipLaunchKernelGGL(k_adapter_transpose, dim3((unsigned)(T.a[0].blocks + T.a[1].blocks)), dim3(256), 0, s, T);
    return launched();
}

lpq_status adapters_forward_shape(const Adapters& P) {
    const lpq_status st = adapters_shape(P);
    if (st != LPQ_OK) return st;
    return expand_shape(P, P.N, P.tokens).blocks > max_groups(64 * kExpandWaves) ? LPQ_ERR_SHAPE : LPQ_OK;
}
lpq_status adapters_backward_shape(const Adapters& P) {
    const lpq_status st = adapters_shape(P);
    if (st != LPQ_OK) return st;
    const AdapterTransposePair T = transpose_pair(P, nullptr, nullptr, nullptr, nullptr);
    if ((int64_t)T.a[0].blocks + T.a[1].blocks > max_groups(256)) return LPQ_ERR_SHAPE;
    return expand_shape(P, P.K, P.tokens).blocks > max_groups(64 * kExpandWaves) ? LPQ_ERR_SHAPE : LPQ_OK;
}

int64_t whole_lines(int64_t n) { return ceil_div(n, 256) * 256; }

}  // namespace

extern "C" {

int64_t lpq_adapters_workspace(int64_t tokens, int64_t capacity, int32_t groups, int32_t rank, int64_t N, int64_t K) {
    const Adapters P{tokens, capacity, groups, rank, N, K};
    return adapters_forward_shape(P) == LPQ_OK ? shrink_bytes(P, K) : 0;
}

lpq_status lpq_adapters(const uint16_t* x, const uint16_t* A, const uint16_t* B, const float* scale, const int32_t* offsets,
                        const int32_t* rows, const int32_t* src, int64_t tokens, int64_t capacity, int32_t groups, int32_t rank,
                        int64_t N, int64_t K, const uint16_t* base, uint16_t* y, void* workspace, int64_t workspace_bytes, void* stream) {
    const Adapters P{tokens, capacity, groups, rank, N, K};
    lpq_status st = adapters_forward_shape(P);
    if (st != LPQ_OK) return st;
    if (!x || !A || !B || !offsets || !rows || !src || !y || !workspace) return LPQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(base, 16) || !aligned(y, 16) || !aligned(workspace, 16) ||
        !aligned(scale, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(src, 4))
        return LPQ_ERR_ALIGN;
    const int64_t need = shrink_bytes(P, K), factor = 2 * (int64_t)groups * rank;
    if (workspace_bytes < need) return LPQ_ERR_ARG;
    if (any_overlap({range(y, 2 * tokens * N), range(workspace, need)},
                    {range(x, 2 * tokens * K), range(A, factor * K), range(B, factor * N), range(scale, 4 * groups),
                     range(offsets, 4 * (groups + 1)), range(rows, 4 * tokens), range(src, 4 * capacity),
                     range(base == y ? nullptr : base, 2 * tokens * N)}))
        return LPQ_ERR_ARG;
    const Routing R{offsets, groups, (int32_t)capacity};
    const hipStream_t s = (hipStream_t)stream;
    float* u = static_cast<float*>(workspace);
    if ((st = adapter_shrink(P, R, {x, A, u, K}, {}, src, s)) != LPQ_OK) return st;
    return adapter_expand(P, R, u, shrink_splits(P, K), B, N, scale, rows, src, base, y, s);
}

int64_t lpq_adapters_backward_workspace(int64_t tokens, int64_t capacity, int32_t groups, int32_t rank, int64_t N, int64_t K) {
    const Adapters P{tokens, capacity, groups, rank, N, K};
    if (adapters_backward_shape(P) != LPQ_OK) return 0;
    const int64_t factor = 2 * (int64_t)groups * rank;
    return whole_lines(factor * K) + whole_lines(factor * N) + whole_lines(shrink_bytes(P, K)) + whole_lines(shrink_bytes(P, N)) +
           2 * whole_lines(planes_bytes(P)) + whole_lines(grad_bytes(P, K)) + grad_bytes(P, N);
}

lpq_status lpq_adapters_backward(const uint16_t* dy, const uint16_t* x, const uint16_t* A, const uint16_t* B, const float* scale,
                                 const int32_t* offsets, const int32_t* rows, const int32_t* src, int64_t tokens, int64_t capacity,
                                 int32_t groups, int32_t rank, int64_t N, int64_t K, const uint16_t* dres, uint16_t* dx, float* dA,
                                 float* dB, int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
    const Adapters P{tokens, capacity, groups, rank, N, K};
    lpq_status st = adapters_backward_shape(P);
    if (st != LPQ_OK) return st;
    if (!dy || !x || !A || !B || !offsets || !rows || !src || !dx || !dA || !dB || !workspace) return LPQ_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(dres, 16) || !aligned(dx, 16) ||
        !aligned(dA, 16) || !aligned(dB, 16) || !aligned(workspace, 16) || !aligned(scale, 4) || !aligned(offsets, 4) ||
        !aligned(rows, 4) || !aligned(src, 4))
        return LPQ_ERR_ALIGN;
    const int64_t need = lpq_adapters_backward_workspace(tokens, capacity, groups, rank, N, K), factor = 2 * (int64_t)groups * rank;
    if (workspace_bytes < need) return LPQ_ERR_ARG;
    if (any_overlap({range(dx, 2 * tokens * K), range(dA, 2 * factor * K), range(dB, 2 * factor * N), range(workspace, need)},
                    {range(dy, 2 * tokens * N), range(x, 2 * tokens * K), range(A, factor * K), range(B, factor * N),
                     range(scale, 4 * groups), range(offsets, 4 * (groups + 1)), range(rows, 4 * tokens), range(src, 4 * capacity),
                     range(dres == dx ? nullptr : dres, 2 * tokens * K)}))
        return LPQ_ERR_ARG;
    const Routing R{offsets, groups, (int32_t)capacity};
    const hipStream_t s = (hipStream_t)stream;
    uint8_t* at = static_cast<uint8_t*>(workspace);
    auto take = [&](int64_t bytes) {
        uint8_t* p = at;
        at += whole_lines(bytes);
        return p;
    };
    uint16_t* At = reinterpret_cast<uint16_t*>(take(factor * K));   // [groups, K, rank]
    uint16_t* Bt = reinterpret_cast<uint16_t*>(take(factor * N));   // [groups, rank, N]
    float* u = reinterpret_cast<float*>(take(shrink_bytes(P, K)));
    float* du = reinterpret_cast<float*>(take(shrink_bytes(P, N)));
    uint16_t* planes[2] = {reinterpret_cast<uint16_t*>(take(planes_bytes(P))), reinterpret_cast<uint16_t*>(take(planes_bytes(P)))};
    float* part_a = reinterpret_cast<float*>(take(grad_bytes(P, K)));
    float* part_b = reinterpret_cast<float*>(at);
    const int32_t parts = shrink_splits(P, K), dparts = shrink_splits(P, N);
    if ((st = adapter_transpose(transpose_pair(P, A, At, B, Bt), s)) != LPQ_OK) return st;
    if ((st = adapter_shrink(P, R, {x, A, u, K}, {dy, Bt, du, N}, src, s)) != LPQ_OK) return st;
    const AdapterPlanesArgs planes_args{{du, u}, {planes[0], planes[1]}, {dparts, parts}, rank, (int32_t)planes_pitch(P)};
    hipLaunchKernelGGL(k_adapter_planes, dim3((unsigned)(planes_pitch(P) / 64), (unsigned)ceil_div(rank, 16), 2), dim3(256), 0, s, planes_args, R);
    if ((st = launched()) != LPQ_OK) return st;
    const Gradient gradients[2] = {{x, K, planes[0], part_a, dA, 0}, {dy, N, planes[1], part_b, dB, 1}};
    if ((st = adapter_grad(P, R, gradients, scale, src, accumulate, s)) != LPQ_OK) return st;
    return adapter_expand(P, R, du, dparts, At, K, scale, rows, src, dres, dx, s);
}

lpq_status lpq_mx_matmul_routed(const uint8_t* a, const uint8_t* ae, int a_format, const uint8_t* b, const uint8_t* be, int b_format,
                                const int32_t* offsets, int32_t groups, int64_t capacity, int64_t N, int64_t K, void* y, int y_type,
                                void* stream) {
    const int64_t most = int64_t(1) << 40;
    if (groups <= 0 || groups > kRouteMaxGroups || capacity <= 0 || N <= 0 || K <= 0 || K % 32) return LPQ_ERR_SHAPE;
    if (capacity > kRouteMaxRows || N > kRouteMaxRows || K > kRouteMaxRows) return LPQ_ERR_SHAPE;
    if (capacity > most / N || capacity > most / K || N > most / K / groups) return LPQ_ERR_SHAPE;
    const lpq_status st = check_routed({a, ae, b, be, a_format, b_format, offsets, groups, capacity, groups * N, N, K, capacity * N, y, y_type});
    if (st != LPQ_OK) return st;
    const MatmulArgs A{a, ae, b, be, y, (int32_t)capacity, (int32_t)N, (int32_t)K, y_type == LPQ_F32};
    const Routing R{offsets, groups, (int32_t)capacity};
    const hipStream_t s = (hipStream_t)stream;
    if (a_format == LPQ_MXFP4) return b_format == LPQ_MXFP4 ? mx_matmul_routed<true, true>(A, R, s) : mx_matmul_routed<true, false>(A, R, s);
    return b_format == LPQ_MXFP4 ? mx_matmul_routed<false, true>(A, R, s) : mx_matmul_routed<false, false>(A, R, s);
}

lpq_status lpq_mx_matmul_routed_dw(const uint8_t* a, const uint8_t* ae, int a_format, const uint8_t* b, const uint8_t* be,
                                   int b_format, const int32_t* offsets, int32_t groups, int64_t M, int64_t N, int64_t capacity,
                                   void* y, int y_type, void* stream) {
    const int64_t most = int64_t(1) << 40;
    if (groups <= 0 || groups > kRouteMaxGroups || M <= 0 || N <= 0 || capacity <= 0 || capacity % 32) return LPQ_ERR_SHAPE;
    if (capacity > kRouteMaxRows || M > kRouteMaxRows || N > kRouteMaxRows) return LPQ_ERR_SHAPE;
    if (M > most / capacity || N > most / capacity || M > most / N / groups) return LPQ_ERR_SHAPE;
    const lpq_status st = check_routed({a, ae, b, be, a_format, b_format, offsets, groups, M, N, N, capacity, groups * M * N, y, y_type});
    if (st != LPQ_OK) return st;
    const MatmulArgs A{a, ae, b, be, y, (int32_t)M, (int32_t)N, (int32_t)capacity, y_type == LPQ_F32};
    const Routing R{offsets, groups, (int32_t)capacity};
    const hipStream_t s = (hipStream_t)stream;
    if (a_format == LPQ_MXFP4) return b_format == LPQ_MXFP4 ? mx_matmul_routed_dw<true, true>(A, R, s) : mx_matmul_routed_dw<true, false>(A, R, s);
    return b_format == LPQ_MXFP4 ? mx_matmul_routed_dw<false, true>(A, R, s) : mx_matmul_routed_dw<false, false>(A, R, s);
}

int64_t lpq_route_capacity(int64_t pairs, int32_t groups, int32_t align) { return route_capacity(pairs, groups, align); }

int64_t lpq_route_plan_workspace(int64_t pairs, int32_t groups) {
    if (route_capacity(pairs, groups, 1) == 0) return 0;
    const int64_t runs = plan_runs(pairs);
    return runs == 1 ? 0 : 4 * runs * groups;
}

lpq_status lpq_route_plan(const void* ids, int id_bytes, int64_t pairs, int32_t groups, int32_t align, int32_t* offsets,
                          int32_t* rows, int32_t* src, int64_t capacity, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t least = route_capacity(pairs, groups, align), need = lpq_route_plan_workspace(pairs, groups);
    if (least == 0 || capacity < least || capacity > kRouteMaxRows) return LPQ_ERR_SHAPE;
    if (!ids || !offsets || !rows || !src || (need && !workspace)) return LPQ_ERR_NULL;
    if ((id_bytes != 4 && id_bytes != 8) || workspace_bytes < need) return LPQ_ERR_ARG;
    if (!aligned(ids, id_bytes) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(src, 4) || !aligned(workspace, 4))
        return LPQ_ERR_ALIGN;
    if (any_overlap({range(offsets, 4 * (groups + 1)), range(rows, 4 * pairs), range(src, 4 * capacity), range(workspace, need)},
                    {range(ids, id_bytes * pairs)}))
        return LPQ_ERR_ARG;
    const PlanArgs A{ids, pairs, 0, groups, align, offsets, rows, src, capacity, static_cast<int32_t*>(workspace)};
    return id_bytes == 4 ? route_plan<int32_t>(A, (hipStream_t)stream) : route_plan<int64_t>(A, (hipStream_t)stream);
}

lpq_status lpq_route_gather(const uint16_t* x, int64_t tokens, int64_t N, const int32_t* rows, int64_t k, const int32_t* src,
                            int64_t capacity, uint16_t* y, void* stream) {
    return route_gather<ROW_BF16>(x, tokens, N, rows, k, src, capacity, y, nullptr, stream);
}

lpq_status lpq_route_gather_mxfp8(const uint16_t* x, int64_t tokens, int64_t N, const int32_t* rows, int64_t k, const int32_t* src,
                                  int64_t capacity, uint8_t* q, uint8_t* e, void* stream) {
    return route_gather<ROW_FP8>(x, tokens, N, rows, k, src, capacity, q, e, stream);
}

lpq_status lpq_route_gather_mxfp4(const uint16_t* x, int64_t tokens, int64_t N, const int32_t* rows, int64_t k, const int32_t* src,
                                  int64_t capacity, uint8_t* p, uint8_t* e, void* stream) {
    return route_gather<ROW_FP4>(x, tokens, N, rows, k, src, capacity, p, e, stream);
}

lpq_status lpq_route_combine(const uint16_t* y, int64_t capacity, int64_t N, const int32_t* rows, int64_t tokens, int64_t k,
                             const float* weights, const uint16_t* residual, uint16_t* out, void* stream) {
    const lpq_status st = route_shape(tokens, k, capacity, N);
    if (st != LPQ_OK) return st;
    const int64_t blocks = ceil_div(tokens * (N / 8), kRouteThreads);
    if (blocks > max_groups(kRouteThreads)) return LPQ_ERR_SHAPE;
    if (!y || !rows || !out) return LPQ_ERR_NULL;
    if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(rows, 4) || !aligned(weights, 4)) return LPQ_ERR_ALIGN;
    if (any_overlap({range(out, 2 * tokens * N)},   // out may be the residual itself: a thread reads what it writes first
                    {range(y, 2 * capacity * N), range(rows, 4 * tokens * k), range(weights, 4 * tokens * k),
                     range(residual == out ? nullptr : residual, 2 * tokens * N)}))
        return LPQ_ERR_ARG;
    const CombineArgs A{y, rows, weights, residual, out, tokens, capacity, (int32_t)k, (int32_t)N};
    hipLaunchKernelGGL(k_route_combine, dim3((unsigned)blocks), dim3(kRouteThreads), 0, (hipStream_t)stream, A);
    return launched();
}

lpq_status lpq_route_combine_backward(const uint16_t* dout, const uint16_t* y, int64_t capacity, int64_t N, const int32_t* rows,
                                      const int32_t* src, int64_t tokens, int64_t k, const float* weights, uint16_t* dy,
                                      float* dweights, void* stream) {
    const lpq_status st = route_shape(tokens, k, capacity, N);
    if (st != LPQ_OK) return st;
    const bool wide = N > 512;   // one wave to a row of up to 64 vectors
    const int threads = wide ? 256 : 64;
    const int64_t pad = ceil_div(capacity, kPadRows), blocks = pad + tokens;
    if (blocks > max_groups(threads)) return LPQ_ERR_SHAPE;
    if (!dout || !rows || !src || !dy || (dweights && !y)) return LPQ_ERR_NULL;
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(rows, 4) || !aligned(src, 4) || !aligned(weights, 4) ||
        !aligned(dweights, 4))
        return LPQ_ERR_ALIGN;
    if (any_overlap({range(dy, 2 * capacity * N), range(dweights, 4 * tokens * k)},
                    {range(dout, 2 * tokens * N), range(dweights ? y : nullptr, 2 * capacity * N), range(rows, 4 * tokens * k),
                     range(src, 4 * capacity), range(weights, 4 * tokens * k)}))
        return LPQ_ERR_ARG;
    const CombineGradArgs A{dout, dweights ? y : nullptr, rows, src, weights, dy, dweights, tokens, capacity, (int32_t)k, (int32_t)N,
                            (int32_t)pad};
    if (wide) hipLaunchKernelGGL(k_route_combine_grad<256>, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, A);
    else hipLaunchKernelGGL(k_route_combine_grad<64>, dim3((unsigned)blocks), dim3(64), 0, (hipStream_t)stream, A);
    return launched();
}

}  // extern "C"
