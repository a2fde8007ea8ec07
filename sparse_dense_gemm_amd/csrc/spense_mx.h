// Declarations shared by the host code and the HIP kernels of the microscaled
// 4-bit (mx4) layers, the experts' layers and the router.
//
// mx4: e2m1 codes (sign, two exponent bits, one fraction bit: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6), 32 consecutive columns of a row sharing one power of two,
// stored as its exponent plus 127 in a byte (255: the block is NaN).
//
// Packed weights.  An expert's N rows are padded to row tiles of 16 (the rows
// of a matrix instruction), K to units of 128 columns.  Per row tile:
//   mx4:  [units][64 lanes][16 B], lane l holding the 32 codes of row l % 16,
//         columns 32 (l / 16) .. + 31 of the unit; then
//         [ceil(units / 4)][64 lanes][4 B], byte u the exponent byte of unit
//         4 i + u for the same row and columns;
//   bf16: [units][4 steps][64 lanes][16 B], lane l holding row l % 16, columns
//         32 step + 8 (l / 16) .. + 7 of the unit.
// So a lane's 16 bytes are its operand of a matrix instruction as they are
// (mx4 x mx4: one 16x16x128 product per unit; bf16: one 16x16x32 per step; mx4
// x bf16: dword j, eight columns of each lane, widened, meets the same columns
// of the activations), and a wave streams whole kilobytes.  Padding rows and
// columns hold zeros with exponent byte 127.  A gate/up layer (glu) of 2I rows
// is packed as pairs (gate i, up i).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/spense.h"
#include "spense_internal.h"

namespace spense {

enum : int32_t { DT_MX4 = 3 };

constexpr int kMxBlock = 32;   // columns that share an exponent
constexpr int kUnitK = 128;    // columns of a packed unit
constexpr int kStageBytes = 256;  // bytes of one activation row in a stage of the product kernel

__host__ __device__ inline int64_t mx_units(int64_t K) { return (K + kUnitK - 1) / kUnitK; }

struct ExpertsDesc {
  int64_t E, N, K;     // experts; rows (2I of a gate/up layer) and columns of each
  int32_t wdtype;      // DT_BF16 or DT_MX4
  int32_t glu;         // 1: write silu(gate) * up, N / 2 columns
  int64_t NT;          // row tiles of an expert
  int64_t NU;          // units of a row tile
  int64_t tile_bytes;  // bytes of a row tile
  int64_t scale_off;   // mx4: offset of the exponent bytes in a row tile
  uint8_t* wpack;      // E * NT * tile_bytes
};

struct ExpertsArgs {
  const uint8_t* X;      // activation rows: bf16 (16-byte aligned rows) or mx4 codes
  const uint8_t* xs;     // mx4 activations: exponent bytes, 16 per row and stage
  int64_t ldx, ldxs;     // bytes from row to row
  int64_t M;             // rows of X
  int64_t xbytes;        // bytes of a row that hold data (a multiple of 16)
  const int32_t* rows;   // X row of each grouped row, or nullptr: X is grouped already
  const int32_t* offsets;  // [E + 1], or nullptr: one expert takes all R rows
  int64_t R;             // grouped rows (capacity)
  void* Y;
  int64_t ldy;
  int32_t ydtype;
  float* ws;             // [splits][NT][R][16] partial sums (splits > 1)
  int32_t* counters;     // [m-tiles * row groups], zero between calls
};

struct ExpertsPlan {
  int config;   // index into the configurations of spense_experts.hip
  int splits;
  int rgroups;  // groups of row tiles, one per workgroup
  int mgroups;  // groups of activation rows (upper bound over the experts)
  int rblock;   // row groups taken together before the next m-group (launch order)
  int run;      // consecutive tiles that one XCD takes; 0: as many as gives every XCD the same
};

// A configuration of the product kernel: waves per workgroup, row tiles per
// wave, m-tiles (16 activation rows), stages in flight.
struct ExpertsShape {
  int waves, r, t, stages;
};
int experts_config_count();
ExpertsShape experts_shape(int config);

// xdtype: DT_BF16 or DT_MX4 (then d.wdtype is DT_MX4)
hipError_t launch_experts(const ExpertsDesc& d, const ExpertsArgs& a, int32_t xdtype, const ExpertsPlan& p,
                          hipStream_t s);
// X [M, K] bf16 (rows by `rows` if given, R of them) as rows of ldo bytes, zeros from K on
hipError_t launch_pad_rows(const void* X, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R, void* out,
                           int64_t ldo, hipStream_t s);

// ---- spense_mx.hip ----
hipError_t launch_mx4_quantize(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, uint8_t* codes,
                               int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t s);
// the product kernel's activations (bf16 X, its R rows by `rows` if given): codes of 64 bytes per unit, exponent
// bytes in lane order, both padded
hipError_t launch_mx4_activations(const void* X, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R,
                                  uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t s);
hipError_t launch_mx4_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t M,
                                 int64_t K, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s);
// W: bf16 [E N, ldw] or mx4 codes [E N, ldw bytes] with scales [E N, lds]
hipError_t launch_pack_experts(const ExpertsDesc& d, const void* W, int64_t ldw, const uint8_t* scales, int64_t lds,
                               hipStream_t s);

// ---- spense_route.hip ----
struct RouteArgs {
  const void* logits;
  int32_t ltype;
  int64_t T, E, ldl;
  int32_t k;
  int32_t renormalize;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* pos;
  int32_t* work;
};
int64_t route_work_bytes(int64_t T, int64_t E);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_combine(const void* O, int32_t otype, int64_t R, int64_t ldo, const int32_t* pos,
                          const float* weights, int64_t T, int64_t k, int64_t N, void* Y, int32_t ydtype, int64_t ldy,
                          hipStream_t s);

// ---- host side (spense_mx_api.cpp); status codes of spense.h ----
struct ExpertsLayer;
int experts_pack(const void* W, int32_t wdtype, const uint8_t* scales, int64_t E, int64_t N, int64_t K, int64_t ldw,
                 int64_t lds, int32_t glu, hipStream_t s, ExpertsLayer** out);
void experts_release(ExpertsLayer* h);
void experts_info(const ExpertsLayer* h, spense_layer_info* info);
const ExpertsDesc& experts_desc(const ExpertsLayer* h);
int experts_run(ExpertsLayer* h, const void* X, int32_t adtype, int64_t M, int64_t ldx, const int32_t* rows,
                const int32_t* offsets, int64_t R, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s);
// records a HIP failure for spense_last_hip_error and returns SPENSE_EHIP (spense_api.cpp)
int report_hip(hipError_t e);

}  // namespace spense
