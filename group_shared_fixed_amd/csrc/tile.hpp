// Matrix-core tiles fed through an LDS ring: operand moves, operand reads and
// the products they feed (softmax loss, 8-bit scoring).
#pragma once

#include "elem.hpp"

namespace haste {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 32x32x16 product, fp32 accumulate.  Lane l supplies A row (l % 32) and B
// column (l % 32), contraction elements 8 (l / 32) .. + 8; lane l holds
// column (l % 32), element e at row 8 (e / 4) + 4 (l / 32) + e % 4.
template <int DT>
__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c)
{
    if constexpr (DT == HASTE_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
}

// An operand tile: T (256 or 128) tile rows by one stage of ST contraction elements.
// Contraction-contiguous operands (TR = false) lie in memory as one row of
// `ld` elements per tile row; row-contiguous ones (TR = true) as one row of
// ld elements per contraction index, with the tile rows along it.
struct Operand {
    const uint16_t* p;
    int64_t ld;
    int64_t rows;     // valid tile-row indices: [0, rows), past it the last one is read again
    int64_t depth;    // valid contraction indices, likewise
    int64_t block = 0;   // BLOCKED (TR = false): elements from one run of 256 contraction indices to the next
};

// Waits until at most N of this wave's moves are in flight and its LDS reads
// are done (vmcnt(N) and lgkmcnt(0), expcnt at its no-wait maximum).
template <int N>
__device__ __forceinline__ void wait_stage()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
// Workgroup barrier without a memory fence (a fence would wait for every
// move in flight); the empty asm statements keep the compiler from moving
// memory accesses across it.
__device__ __forceinline__ void stage_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
typedef __attribute__((address_space(3))) void* lds_ptr;
// One wave's move of 64 x 16 bytes from memory into LDS, from the lanes' src
// to the wave's dst.
__device__ __forceinline__ void move16(const void* src, uint16_t* dst)
{
    __builtin_amdgcn_global_load_lds(src, (lds_ptr)dst, 16, 0, 0);
}

// Moves of one operand tile from memory straight into LDS
// (global_load_lds_dwordx4: a lane's 16 bytes land at the wave's LDS base +
// 16 x lane).  LDS images in 16-byte pieces: TR = false: tile row r, piece
// c (of P = ST / 8) at P r + (c ^ row_swizzle(r)).  TR = true: contraction
// row k, piece c (of T / 8) at (T / 8) k + (c ^ 4 (k % 4)).  Both spread the
// pieces that one operand read touches over the banks; since a lane's place
// in LDS is fixed, the swizzle is in the piece it asks for.
template <int ST>
__device__ __forceinline__ int row_swizzle(int r)
{
    return ST == 64 ? (r >> 1) & 7 : (r >> 2) & 3;
}

template <int T, bool TR, int ST, int THREADS, bool BLOCKED = false>
struct Mover {
    static_assert(!(TR && BLOCKED), "");
    static constexpr int N = T * ST / 8 / THREADS;   // moves per wave and stage
    const char* base;                         // tile's first row (TR: column), contraction index 0
    uint32_t off[N];                          // byte offset of the lane's piece
    int64_t step;                             // TR: bytes per stage; BLOCKED: bytes per block
    uint32_t row[N], pitch;                   // contraction index within the stage, bytes per row
    int64_t depth;

    __device__ __forceinline__ Mover(const Operand& o, int64_t r0, int wave, int lane)
    {
        depth = o.depth;
        pitch = 2 * (uint32_t)o.ld;
        if constexpr (TR) {
            base = reinterpret_cast<const char*>(o.p);
            step = 2 * ST * o.ld;
        } else {
            base = reinterpret_cast<const char*>(o.p + r0 * o.ld);
            step = 2 * o.block;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = 64 * (N * wave + i) + lane;
            if constexpr (TR) {
                const int k = u / (T / 8), c = (u % (T / 8)) ^ (4 * (k & 3));
                int64_t r = r0 + 8 * c;
                r = r < o.rows - 8 ? r : o.rows - 8;
                row[i] = (uint32_t)k;
                off[i] = 2 * (uint32_t)r;
            } else {
                const int r = u / (ST / 8), c = (u % (ST / 8)) ^ row_swizzle<ST>(r);
                const int64_t last = o.rows - 1 - r0;
                row[i] = 8 * (uint32_t)c;
                off[i] = (uint32_t)(r < last ? r : last) * pitch;
            }
        }
    }

    // stage st into buf; pieces past the operand's depth repeat its last one
    __device__ __forceinline__ void move(int st, uint16_t* buf, int wave) const
    {
        const char* b = base;
        if constexpr (TR) b += (int64_t)st * step;
        if constexpr (BLOCKED) b += (int64_t)(st / (256 / ST)) * step + 2 * ST * (st % (256 / ST));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t o;
            if constexpr (TR) {
                const int left = (int)depth - st * ST;
                const uint32_t last = left < ST ? (uint32_t)left - 1 : ST - 1;
                o = off[i] + (row[i] < last ? row[i] : last) * pitch;
            } else if constexpr (BLOCKED) {
                o = off[i] + 2 * row[i];
            } else {
                const uint32_t k = (uint32_t)st * ST + row[i], last = (uint32_t)depth - 8;
                o = off[i] + 2 * (k < last ? k : last);
            }
            move16(b + o, buf + 512 * (N * wave + i));
        }
    }
};

// LDS byte address of a pointer into LDS.
__device__ __forceinline__ uint32_t lds_address(const uint16_t* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint16_t*)p;
}

// Operand fragments of NF x 32 tile rows from row 32 x0 on, contraction step s
// (16 deep).
//
// TR operands are read with the transposing LDS read in groups, each group
// and its wait in one asm block: through the builtin, the compiler (which
// does not see that the read and the moves in flight touch different
// buffers) waits for every move first, and the ring is empty at each stage.
template <int T, bool TR, int ST, int NF>
__device__ __forceinline__ void fragments(const uint16_t* tile, int x0, int s, int lane, u32x4_t (&f)[NF])
{
    static_assert(NF == 2 || NF == 4, "");
    if constexpr (TR) {
        // lane 16 g + 4 rr + cc: contraction row 16 s + 8 (g / 2) + rr (and + 4), piece 4 x + 2 (g % 2) + cc / 2
        const int g = lane >> 4, rr = (lane >> 2) & 3, cc = lane & 3;
        const uint32_t base = lds_address(tile + (16 * s + 8 * (g >> 1) + rr) * T + 8 * (2 * (g & 1) + (cc >> 1)) + 4 * (cc & 1));
        uint32_t p[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i) p[i] = base + 64 * (uint32_t)((x0 + i) ^ rr);
        u32x2_t v[2 * NF];
        if constexpr (NF == 4)
            asm volatile("ds_read_b64_tr_b16 %0, %8\n\t"
                         "ds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
                         "ds_read_b64_tr_b16 %2, %9\n\t"
                         "ds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
                         "ds_read_b64_tr_b16 %4, %10\n\t"
                         "ds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
                         "ds_read_b64_tr_b16 %6, %11\n\t"
                         "ds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]),
                           "=&v"(v[7])
                         : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "n"(8 * T)
                         : "memory");
        else
            asm volatile("ds_read_b64_tr_b16 %0, %4\n\t"
                         "ds_read_b64_tr_b16 %1, %4 offset:%6\n\t"
                         "ds_read_b64_tr_b16 %2, %5\n\t"
                         "ds_read_b64_tr_b16 %3, %5 offset:%6\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
                         : "v"(p[0]), "v"(p[1]), "n"(8 * T)
                         : "memory");
#pragma unroll
        for (int i = 0; i < NF; ++i) f[i] = cat(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            const int r = 32 * (x0 + i) + (lane & 31);
            f[i] = *reinterpret_cast<const u32x4_t*>(tile + r * ST + 8 * ((2 * s + (lane >> 5)) ^ row_swizzle<ST>(r)));
        }
    }
}

// Tile of this workgroup: ids go round-robin over the 8 XCDs, so each XCD is
// dealt one run of neighbouring tiles, whose operands meet in its L2.
__device__ __forceinline__ int64_t dealt_tile(uint32_t b, uint32_t nb)
{
    const uint32_t per = nb / 8;
    return b < per * 8 ? (b & 7) * per + (b >> 3) : b;
}
__device__ __forceinline__ int64_t dealt_tile() { return dealt_tile(blockIdx.x, gridDim.x); }

}  // namespace haste
