// The constants of e4m3 rows: values of 1 byte with an fp32 scale for each
// block of channels.
#pragma once

namespace kda {

constexpr int kScaleBlock = 128;        // channels that share an e4m3 scale
constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;    // a block of zeros still has a scale

}  // namespace kda
