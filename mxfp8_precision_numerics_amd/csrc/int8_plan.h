// Which kernel takes an int8 product, its grid, and the order of the large tiles (int8.hip). Without device code of its own, so
// that a plain C++ compiler reads it too. Internal; not part of the C ABI.
#pragma once
#include <cstdint>

namespace mxq {

constexpr int CUS = 256;                // of the chip
constexpr int MT_M = 64, MT_N = 128;    // rows of A and B in a middle tile
constexpr int LT = 256;                 // rows of A, and of B, in a large tile

// Upper bound of the row tiles of TH rows over ragged groups: every group with rows adds at most one partial tile.
inline int64_t most_row_tiles(int64_t rows, int64_t G, int64_t TH) { return (rows + TH - 1) / TH + (G < rows ? G : rows); }

// Which kernel takes a call, and its grid. The rules are on the rows of A (for each expert, on average) and on sizes that say how
// many workgroups the middle tiles would make; the times are of one call, us, at rows x N x K.
enum : int { INT8_FEW, INT8_WIDE, INT8_MIDDLE, INT8_LARGE };
struct Int8Plan {
    int kind, rows;             // rows of A in a tile
    int wide;                   // 16-row blocks of B in a wide tile
    bool deep;                  // middle tiles: the longer ring
    int64_t blocks;
};

inline Int8Plan int8_plan(int64_t M, int64_t cols, int64_t K, int64_t G, bool swiglu) {
    Int8Plan p{};
    const int64_t groups = G ? G : 1, N = swiglu ? 2 * cols : cols;
    auto count = [&](int64_t th, int64_t tc) {
        const int64_t tn = (cols + tc - 1) / tc, tm = G ? most_row_tiles(M, G, th) : (M + th - 1) / th;
        return tn > 0 && tm > INT64_MAX / tn ? INT64_MAX : tm * tn;
    };
    const int64_t middle = count(MT_M, swiglu ? MT_N / 2 : MT_N), weight = N * K;
    // One dense pass over weights of 96 MB and more (128 MB for up to 32 tokens, 256 MB for up to 16, as fewer tokens leave less
    // to share): wide tiles, where N makes two blocks a CU. Wide and few at 16 x 36864 x 12288: 79 and 90 us, 61 rows 88 and 132;
    // at 32 x 12288 x 12288 32 and 38, 61 rows 40 and 50; but 16 rows 33 and 31, and at 61 x 8192 x 8192 21 and 15.
    if (!G && M > 4 && M <= 128 && N >= 8192 && weight >= (M <= 16 ? 256000000 : M <= 32 ? 128000000 : 96000000)) {
        p.kind = INT8_WIDE;
        p.rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
        const int64_t units = (cols + 15) / 16;
        int64_t best = INT64_MAX;
        for (int k = 1; k <= (swiglu ? 6 : 12); ++k) {
            const int b = swiglu ? 2 * k : k;
            const int64_t cost = ((units + k - 1) / k + 255) / 256 * (b + p.rows / 16);
            if (cost <= best) {
                best = cost;
                p.wide = b;
            }
        }
        p.blocks = count(p.rows, (swiglu ? 8 : 16) * (int64_t)p.wide);
    // Up to 8 rows an expert (64 dense ones), or so few middle tiles that half the CUs had none: the contraction is shared within
    // a workgroup. Few and middle at 100 x 6144 x 2048: 11 and 13 us, 256 x 2048 x 8192 13 and 34, 200 x 6144 x 2048 17 and 14;
    // 64 experts, up to 2048 x 2048 with SwiGLU: 16 rows an expert 65 and 60, 32 86 and 63.
    } else if (M <= (G ? 8 * groups : 64) || middle <= 128) {
        p.kind = INT8_FEW;
        p.rows = M <= 16 * groups ? 16 : M <= 32 * groups ? 32 : 64;
        p.blocks = count(p.rows, p.rows == 16 || swiglu ? 16 : 32);
    // Three middle tiles a CU are as much as the large ones take for one round. Middle and large at 400 x 12288 x 12288: 117 and
    // 118 us, 300 rows 94 and 117, 512 rows 129 and 123, 768 194 and 124, 160 x 36864 x 12288 209 and 141; 64 experts, up to
    // 2048 x 2048 with SwiGLU, 64 rows each (one middle tile) 69 and 76, 72 rows 82 and 77, 88 rows 84 and 73. Neither is near what
    // weights (7.0 TB/s) and operations (3.0 POP/s) need there: 22 to 52 us for 130 to 512 rows of 12288 x 12288, about 41 for the experts.
    } else if (middle >= 768 && (G ? M > 64 * groups : M >= 80)) {
        p.kind = INT8_LARGE;
        p.rows = LT;
        p.blocks = count(LT, swiglu ? LT / 2 : LT);
    // Three stages, two workgroups a CU, while these hold all tiles; two stages, three workgroups, beyond: at 130 x 12288 x 12288
    // 81 and 91 us, at 400 rows 142 and 117.
    } else {
        p.kind = INT8_MIDDLE;
        p.rows = MT_M;
        p.blocks = middle;
        p.deep = middle <= 512;
    }
    return p;
}

// The large tiles: T of them, taken in turn by large_groups() workgroups, each the tiles large_tile(b, T) for b = its own index and
// every large_groups()-th from there. `most` is the plan's count, which offsets that keep the rule never exceed; groups that overlap, as
// offsets that break it may make them, could. So T ends there, and a workgroup's tiles only ever increase: with 256 workgroups (most >= 256)
// b % 8 stays what it is, and with fewer each takes one tile at most.
constexpr int large_groups(int64_t most) { return most < CUS ? (int)most : CUS; }
constexpr int large_tiles(int64_t row_tiles, int tiles_n, int most) {
    return row_tiles * tiles_n < most ? (int)(row_tiles * tiles_n) : most;
}
constexpr int large_tile(int b, int T) {
    const int T8 = T & ~7;
    return b < T8 ? (b & 7) * (T8 >> 3) + (b >> 3) : b;
}

}  // namespace mxq
