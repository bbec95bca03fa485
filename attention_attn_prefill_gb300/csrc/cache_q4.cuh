// The 4-bit paged cache: number format and layout of a record (one page of one KV head).
//
// A group is 64 channels of one token and KV head.  With hi = max(x, 0) and lo = min(x, 0) over the
// group, the scale s is (hi - lo) / 15 rounded up to 4 significant bits, the zero point z is
// rint(-lo / s) and a value's code is c = clamp(rint(x / s) + z, 0, 15); it stands for s * (c - z).
// |c - z| <= 15 has 4 bits and s has 4, so every value is a bf16 number exactly: attention over the
// codes and attention over values read back to bf16 see the same numbers.
//
// Parameter word (16 bits): the upper 12 bits of s as bf16, whose lower 4 bits are zero, and z there.
//
// Record of 17 d bytes, in the order in which the decode kernel's threads (lane = 4 g + t of a warp)
// take it, as wide loads without bank conflicts:
//   [0, 8 d)        K codes, d / 2 bytes a token.  Word (p, t, e, h) holds channels
//                   64 (2 p + e) + 16 t + 8 h .. + 7, channel j of the eight in nibble j, the word
//                   turned left by 3 bits (each code then lies on a bf16's upper mantissa bits after
//                   a rotation by a multiple of 4).  A token's row is written whole.
//   [8 d, 16 d)     V codes.  Word (i, lane, k) = 16-channel block 4 i + k: byte 0 holds token 2 t, byte 1
//                   token 2 t + 8, byte 2 token 2 t + 1, byte 3 token 2 t + 9, each with channels 2 g
//                   (low nibble) and 2 g + 1 of the block.  No byte is shared by two tokens.
//   [16 d, 16.5 d)  K parameter words [16 tokens][d / 64]
//   [16.5 d, 17 d)  V parameter words [16 tokens][d / 64]
#pragma once

#include <cstdint>

namespace attn {
namespace q4 {

constexpr int PAGE = 16;
constexpr int GROUP = 64;

template <int D>
struct Record {
  static constexpr int NG = D / GROUP;         // groups of a row
  static constexpr int PAIR = NG < 2 ? 1 : 2;  // groups whose words a thread holds next to each other
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = 8 * D;
  static constexpr int KP_OFF = 16 * D;
  static constexpr int VP_OFF = 16 * D + D / 2;
  static constexpr int BYTES = 17 * D;
  // word of a K row that holds channels 8 i .. 8 i + 7
  __device__ static int k_word(int i) {
    const int grp = i / 8, t = i % 8 / 2, h = i % 2;
    return (grp / PAIR) * (8 * PAIR) + t * (2 * PAIR) + grp % PAIR * 2 + h;
  }
  // byte of the V codes that holds channels 2 j, 2 j + 1 of a token
  __device__ static int v_byte(int token, int j) {
    const int lane = j % 8 * 4 + token % 8 / 2;
    return (j / 32 * 32 + lane) * 16 + j / 8 % 4 * 4 + token / 8 + 2 * (token % 2);
  }
};

__device__ __forceinline__ uint32_t rotl3(uint32_t w) { return __funnelshift_l(w, w, 3); }

constexpr uint32_t PARAM_NAN = 0x7fc0;  // the group's values read back as NaN

// Scale of a group with maximum hi >= 0 and minimum lo <= 0: the smallest s of 4 significant bits with
// 15 s >= hi - lo.  The difference is rounded up, which a 15 s (8 bits) never falls below for; the
// quotient is taken a little low and 15 s, exact, decides.
__device__ __forceinline__ float make_scale(float hi, float lo) {
  const float span = __fsub_ru(hi, lo);
  const uint32_t bits = (__float_as_uint(span * 0.06666666f) + 0xfffffu) & 0xfff00000u;
  return __uint_as_float(__uint_as_float(bits) * 15.f < span ? bits + 0x100000u : bits);
}

}  // namespace q4
}  // namespace attn
