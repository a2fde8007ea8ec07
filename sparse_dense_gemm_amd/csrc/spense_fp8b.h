// Declarations shared by the host code and the HIP kernels of the layers with
// block-scaled e4m3 weights (fp8b) and of the norms around a block.
//
// fp8b: e4m3 codes; 128 consecutive columns of a row (activations) or of 128
// consecutive rows (weights) share one 32-bit scale.
//
// Packed weights.  An expert's N rows are padded to row tiles of 16 (the rows
// of a matrix instruction), K to units of 128 columns.  Per row tile
//   [units][2 halves][64 lanes][16 B], lane l holding row l % 16, columns
//   64 half + 16 (l / 16) .. + 15 of the unit,
// so a lane's two pieces are its operand of a 16x16x128 product as they are
// (e4m3 activations), and eight codes at a time, widened, its operands of four
// 16x16x32 products (bf16 activations); a wave streams whole kilobytes.
// Padding rows and columns hold zeros.  A gate/up layer (glu) of 2I rows is
// packed as pairs (gate i, up i); gate and up have blocks of their own.
// Scales: per expert [ceil(rows / 128)][units, rounded up to even][2], for 128
// packed rows at a time: those of even and of odd packed rows (the gate's and the
// up projection's; without glu the same).
#pragma once

#include "spense_mx.h"

namespace spense {

constexpr int kFp8Block = 128;  // columns, and rows of a weight matrix, that share a scale
constexpr float kFp8Top = 448.0f;

struct Fp8bDesc : ExpertsDesc {  // wdtype DT_FP8, tile_bytes = NU * 2048
  int64_t SG;                    // groups of 128 packed rows of an expert
  int64_t NUe;                   // units, rounded up to even
  float* scales;                 // E * SG * NUe * 2
};

// Products: bf16 rows; codes on the instruction for codes (Y in bf16); codes widened to bf16 (Y in fp32).
enum Fp8bKind : int32_t { kBf16 = 0, kCodes = 1, kWide = 2 };

struct Fp8bArgs : ExpertsArgs {  // X: bf16 rows, or codes with scales at xs (row stride ldxs bytes)
  Fp8bKind kind;
  int32_t stream;                // 1: weights with the non-temporal hint (configurations of fewer than 8 m-tiles)
};

// The configurations of spense_fp8b_linear.hip.
int fp8b_config_count(Fp8bKind kind);
ExpertsShape fp8b_shape(Fp8bKind kind, int config);
hipError_t launch_fp8b_linear(const Fp8bDesc& d, const Fp8bArgs& a, const ExpertsPlan& p, hipStream_t s);

// ---- spense_fp8b.hip ----
// rows: 1 or 128
hipError_t launch_fp8b_quantize(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, int rows,
                                uint8_t* codes, int64_t ldc, float* scales, int64_t lds, hipStream_t s);
hipError_t launch_fp8b_dequantize(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int rows,
                                  int64_t M, int64_t K, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s);
// the product kernel's activations: bf16 X (its R rows by `rows` if given) quantised, codes 0 from K up to whole
// units; or codes and scales that are there already, in that layout
hipError_t launch_fp8b_activations(const void* X, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R,
                                   uint8_t* codes, int64_t ldc, float* scales, int64_t lds, hipStream_t s);
hipError_t launch_fp8b_lay_out(const uint8_t* X, int64_t ldx, const float* sx, int64_t lds_in, int64_t M, int64_t K,
                               const int32_t* rows, int64_t R, uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                               hipStream_t s);
// W [E N, ldw] codes; scales [E * blocks, lds], blocks = ceil(N / 128), or 2 ceil(N / 2 / 128) with glu
hipError_t launch_fp8b_pack(const Fp8bDesc& d, const uint8_t* W, int64_t ldw, const float* scales, int64_t lds,
                            hipStream_t s);

// ---- spense_norm.hip ----
hipError_t launch_block_norm(const spense_norm& n, hipStream_t s);

}  // namespace spense
