// A paged cache's rows as a tensor-core operand: tiles of 128 keys in 16 bits
// in shared memory, in blocks of 64 columns in the 128-byte swizzle.
#pragma once

#include "paged_attn.cuh"
#include "tc.cuh"

namespace dflash {

// The lanes of a warp over rows of CH places of 16 bytes: which row and place of an instruction's 32 / CH rows is a
// lane's.  e2m1 codes, whose places become four chunks, have a row a lane first: lanes of a quarter warp then store one
// chunk of eight rows, which are in different banks; e4m3 codes a place first, and the upper half's chunks in the other order.
template <int CB, int HD>
struct TileLanes {
    static constexpr int CH = HD * CB / 128, RPI = 32 / CH;
    static DF_DEV int row(int lane) { return CB == 4 ? lane % RPI : lane / CH; }
    static DF_DEV int place(int lane) { return CB == 4 ? lane / RPI : lane % CH; }
};
// Sixteen bytes of codes (place `ch` of row `key`: 16 e4m3 or 32 e2m1 codes) as f16 (exact) in a tile at dst.  `scales`:
// an e2m1 place's two block scales, e4m3 bytes (code times block scale is exact too: 2 bits times 4).
template <int CB, int HD>
DF_DEV void tile_place(unsigned char* dst, int key, int ch, const uint4& x, uint32_t scales) {
    constexpr int CH = HD * CB / 128;  // places of a row
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (CB == 4) {
        const uint32_t s2 = e4m3x2_f16x2(scales);
        // chunks 4 ch .. of the row: they differ in bits 4 and 5 of the swizzled place
        const uint32_t at = smem_addr(dst) + (ch >> 1) * (kPaTile * 128) + at_swz(key, 4 * (ch & 1));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // a word: eight columns of one block
            const uint32_t s1 = __byte_perm(s2, 0, j >> 1 ? 0x3232 : 0x1010);
            uint32_t y[4];
            e2m1x8_f16x8(w[j], y);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at ^ (16 * j)), "r"(mul_f16x2(y[0], s1)), "r"(mul_f16x2(y[1], s1)),
                         "r"(mul_f16x2(y[2], s1)), "r"(mul_f16x2(y[3], s1))
                         : "memory");
        }
    } else {
        uint32_t y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) e4m3x4_f16x4(w[j], y[2 * j], y[2 * j + 1]);
        const bool flip = ch >= CH / 2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int up = flip ? 1 - j : j, chunk = 2 * ch + up;
            const uint4 v = up ? make_uint4(y[4], y[5], y[6], y[7]) : make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(dst + (chunk >> 3) * (kPaTile * 128) + at_swz(key, chunk & 7)) = v;
        }
    }
}

// The lane that issues a warp's tcgen05 operations: under this branch the compiler keeps their operands in uniform
// registers (an MMA of M 128 and N 64 then goes out every 32 clocks, its own time; predicated on a lane's number it took
// 59, under a branch on it longer).  The same lane each time.
DF_DEV bool pt_elect() {
    uint32_t on;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(on));
    return on != 0;
}
DF_DEV void pt_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

}  // namespace dflash
