// Generated by fit_exp2_poly.py (minimax degree 5 for 2^f, f in [-1/2, 1/2],
// relative error 2.114e-07 after rounding to fp32).  Do not edit by hand.
#pragma once
namespace ta {
constexpr float kExp2P5C0 = 0x1.0000020000000p+0f;  // 1.00000012
constexpr float kExp2P5C1 = 0x1.62e4280000000p-1f;  // 0.693146944
constexpr float kExp2P5C2 = 0x1.ebf9180000000p-3f;  // 0.240221202
constexpr float kExp2P5C3 = 0x1.c6b6e40000000p-5f;  // 0.0555071309
constexpr float kExp2P5C4 = 0x1.3d0c520000000p-7f;  // 0.00967554096
constexpr float kExp2P5C5 = 0x1.5c08e60000000p-10f;  // 0.00132764725
constexpr float kExp2Poly5RelErr = 2.114046e-07f;
}  // namespace ta
