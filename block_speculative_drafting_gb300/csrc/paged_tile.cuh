// A paged cache's rows as a tensor-core operand: tiles of 128 keys in 16 bits
// in shared memory, in blocks of 64 columns in the 128-byte swizzle.
#pragma once

#include "paged_attn.cuh"
#include "tc.cuh"

namespace dflash {

// Sixteen bytes of codes (place `ch` of row `key`: 16 e4m3 or 32 e2m1 codes) as f16 (exact) in a tile at dst.  `scales`:
// an e2m1 place's two block scales, e4m3 bytes (code times block scale is exact too: 2 bits times 4).
// Places of a row's upper half write their chunks in another order: other banks.
template <int CB, int HD>
DF_DEV void tile_place(unsigned char* dst, int key, int ch, const uint4& x, uint32_t scales) {
    constexpr int CH = HD * CB / 128;  // places of a row
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    auto put = [&](int chunk, const uint4& v) {
        *reinterpret_cast<uint4*>(dst + (chunk >> 3) * (kPaTile * 128) + at_swz(key, chunk & 7)) = v;
    };
    if constexpr (CB == 4) {
        const uint32_t s2 = e4m3x2_f16x2(scales);
        const int flip = ch >= CH / 2 ? 2 : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // a word: eight columns of one block
            const int up = j ^ flip;
            const uint32_t word = flip ? w[j ^ 2] : w[j], s1 = __byte_perm(s2, 0, (up >> 1) ? 0x3232 : 0x1010);
            uint32_t y[4];
            e2m1x8_f16x8(word, y);
            put(4 * ch + up, make_uint4(mul_f16x2(y[0], s1), mul_f16x2(y[1], s1), mul_f16x2(y[2], s1), mul_f16x2(y[3], s1)));
        }
    } else {
        uint32_t y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) e4m3x4_f16x4(w[j], y[2 * j], y[2 * j + 1]);
        const bool flip = ch >= CH / 2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int up = flip ? 1 - j : j;
            put(2 * ch + up, up ? make_uint4(y[4], y[5], y[6], y[7]) : make_uint4(y[0], y[1], y[2], y[3]));
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
