// Pieces shared by the matrix-product kernels (gemm.hip, int8.hip): the search for a row group's tile, buffer resources and
// asynchronous copies from global memory to LDS. Internal; not part of the C ABI.
#pragma once
#include "mxq_device.h"

namespace mxq {

typedef int v4i __attribute__((ext_vector_type(4)));

// Row-grouped GEMMs: the expert group that holds row tile t (tiles of TH rows, numbered group by group, each group's
// rows [off[q], off[q+1]) clamped to [0, M) and cut into ceil(rows / TH) tiles). Each wave scans 64 groups at a time:
// lane l loads group base + l's offsets, a wave prefix sum of the tile counts finds the group, so a workgroup pays one
// round of loads per 64 groups instead of a dependent load per group. grp = -1 when t lies past the last tile.
struct RowTile {
    int64_t grp, lo, hi;      // group, first row of the tile, end of the group's rows
};

template <int TH>
__device__ __forceinline__ RowTile find_row_tile(const int64_t* offsets, int64_t G, int64_t M, int64_t t) {
    const int lane = threadIdx.x & 63;
    RowTile r{-1, 0, 0};
    int64_t before = 0;                          // tiles of the groups already scanned
    for (int64_t base = 0; base < G; base += 64) {
        const int64_t q = base + lane;
        int64_t a0 = 0, a1 = 0;
        int nt = 0;
        if (q < G) {
            a0 = offsets[q];
            a1 = offsets[q + 1];
            a0 = a0 < 0 ? 0 : (a0 > M ? M : a0);
            a1 = a1 < a0 ? a0 : (a1 > M ? M : a1);
            nt = (int)((a1 - a0 + TH - 1) / TH);
        }
        int incl = nt;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off, 64);
            if (lane >= off) incl += v;
        }
        const uint64_t hit = __ballot(before + incl > t);
        if (hit) {
            const int L = __ffsll((unsigned long long)hit) - 1;
            const int64_t excl = before + __shfl(incl - nt, L, 64);
            r.grp = base + L;
            r.lo = __shfl(a0, L, 64) + (t - excl) * TH;
            r.hi = __shfl(a1, L, 64);
            return r;
        }
        before += __shfl(incl, 63, 64);
    }
    return r;
}

// Raw buffer resource (base, stride 0, 2^31 - 1 bytes, raw untyped access) for a workgroup-uniform address. The
// address is moved to scalar registers explicitly: values derived from the tile index are computed with vector
// instructions, and the descriptor must live in scalar registers.
// With `records` set, accesses at or past that many bytes from the base are out of range: loads return zero and
// nothing outside the buffer is touched.
__device__ __forceinline__ v4i buffer_rsrc(const void* p, uint32_t records = 0x7FFFFFFFu) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return v4i{(int)lo, (int)(hi & 0xFFFFu), (int)__builtin_amdgcn_readfirstlane(records), 0x00020000};
}

// LDS offset (the low 32 bits of a shared-aperture address) of an LDS location, made wave-uniform.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(p));
}

// Asynchronous copy global -> LDS: each lane reads BYTES (16 or 4) at base + voff + soff and the wave's results land
// in consecutive slots starting at LDS offset `lds` (M0). Written as inline assembly on purpose: the compiler does
// not then treat the copy as an LDS write, so LDS reads of other stages are not made to wait for it. The kernel
// orders copies itself (wait_copies_barrier): a stage is read only after its copies have completed on every wave,
// and a buffer is refilled only after every wave has finished reading it.
template <int BYTES>
__device__ __forceinline__ void dma_to_lds(v4i rsrc, uint32_t lds, int voff, int soff) {
    if constexpr (BYTES == 16)
        asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds"
                     :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
    else
        asm volatile("buffer_load_dword %0, %1, %2 offen lds"
                     :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
}

// Wait until at most N of this wave's copies are still outstanding (vector-memory counter, which retires in issue
// order) and all its LDS reads have returned, then join the workgroup barrier. One asm statement with a memory
// clobber, so the compiler keeps LDS accesses on their side of it.
template <int N>
__device__ __forceinline__ void wait_copies_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}

}  // namespace mxq
