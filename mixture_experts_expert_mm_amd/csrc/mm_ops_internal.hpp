// Internal interfaces of the router, the few-token layer, the block-scaled
// product, the token sort, the activation and the 8-bit integer product
// (mm_router.hip, mm_few.hip, mm_block.hip, mm_sort.hip, mm_swiglu.hip,
// mm_int8.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/megamoe.h"

namespace mm {

// ------------------------------------------------------------------ router
struct RouterArgs {
  const void* x;             // bf16 [T][H]
  const void* w;             // bf16 [E][H]
  const float* bias;         // [E] or null
  const int8_t* active;      // [T] or null
  int32_t* ids;              // [T][K]
  float* weights;            // [T][K]
  float* part;               // ws: [KS][T][Ep] partial scores
  float* xnorm;              // ws: [KS][T] partial |x|^2
  float* xmost;              // ws: [KS][ceil(E / EB)][T] largest partial sum of a token and EB experts
  float* wnorm;              // ws: [KS][Ep] partial |w|^2
  int64_t T;
  int H, E, K, Ep, KS, EB;
  int scoring, renormalize;
  float scale;
  // error of a float32 score in units of 2^-24: of its largest partial sums, of |x| |w| (launch_router_select)
  float of_sums, of_products;
};
struct RouterShape {
  int wide;                  // 0: 16 x 16 a wave; 1: 64 tokens x 64 experts a wave; 2: tiles of 128 x 256 through LDS; 3: of 256 x 256
  int ks;                    // slices of the hidden dimension over workgroups
  int ep;                    // padded experts of a row of partial scores
  int eb;                    // experts of a workgroup
};
RouterShape router_shape(int64_t T, int H, int E);
hipError_t launch_router_scores(const RouterArgs& a, hipStream_t s);
hipError_t launch_router_select(const RouterArgs& a, hipStream_t s);

// --------------------------------------------------------- few-token layer
struct FewArgs {
  const void* x;             // bf16 [T][H]
  const int32_t* ids;        // [T][K]
  const float* weights;      // [T][K]
  const int8_t* active;      // [T] or null
  const uint8_t* w1;         // [E+S][2I][H], gate and up rows interleaved by 32
  const float* s1;           // [E+S][2I], or [E+S][2I/128][H/128], formula order
  const uint8_t* w2;         // [E+S][H][I]
  const float* s2;           // [E+S][H], or [E+S][H/128][I/128]
  uint16_t* a;               // ws: [planes][T*(K+S)][I] bf16 parts of A
  float* slot;               // ws: [T*(K+S)][H] gate-weighted contributions (few_slots)
  void* y;                   // [T][H]
  int T, H, I, E, K, S;
  int format, y_f32;
  float clamp;               // +inf: none
};
// whether Linear2 takes slots of the workspace
bool few_slots(int64_t T, int y_f32);
hipError_t launch_few_l1(const FewArgs& a, int num_cus, hipStream_t s);
hipError_t launch_few_l2(const FewArgs& a, int num_cus, hipStream_t s);

// ---------------------------------------------------- block-scaled product
struct BlockArgs {
  const uint8_t* a;          // e4m3 [M][K]
  const float* as;           // [M][K/128]
  const void* x;             // bf16 [M][K] (quantised on the way), or null
  const uint8_t* b;          // e4m3 [G][N][K]
  const float* bs;           // [G][ceil(N/128)][K/128]
  const int32_t* offsets;    // [G] first row of each group, or null (one group of M rows)
  const int32_t* counts;     // [G] rows of each group
  void* y;                   // bf16 [M][N]
  int64_t M;
  int64_t m_first;           // first row of the streaming units (rows before it: the large tiles)
  int N, K, G;
};
hipError_t launch_block_quantize(const void* x, int64_t rows, int cols, uint8_t* q, float* s, hipStream_t st);
// whether launch_block_gemm holds the rows in LDS, and whether it then quantises a.x on the way (a.a and a.as unused)
bool block_in_lds(const BlockArgs& a);
bool block_from_x(const BlockArgs& a);
hipError_t launch_block_gemm(const BlockArgs& a, int num_cus, hipStream_t s);

// -------------------------------------------------------------- token sort
struct SortArgs {
  const int32_t* ids;        // [T][K]
  const int8_t* active;      // [T] or null
  int32_t* counts;           // [E]
  int32_t* offsets;          // [E+1]
  int32_t* row_of_route;     // [T*K]
  int32_t* route_of_row;     // [T*K]
  const uint8_t* x;          // [T][row_bytes], or null
  uint8_t* rows;             // [T*K][row_bytes], or null
  int32_t* hist;             // ws: [chunks][E]
  int64_t T, R, row_bytes;
  int E, K, chunk, chunks;
};
int sort_chunk(int64_t routes);
// whether launch_sort_few does it all (order and rows); else launch_sort_order, then launch_sort_rows
bool sort_in_one(int64_t routes, int64_t topk);
hipError_t launch_sort_few(const SortArgs& a, hipStream_t s);
hipError_t launch_sort_order(const SortArgs& a, hipStream_t s);
hipError_t launch_sort_rows(const SortArgs& a, hipStream_t s);

struct CombineTokensArgs {
  const void* rows;          // [T*K][H]
  const int32_t* row_of_route;
  const int32_t* offsets;    // [E+1] (backward)
  const float* weights;      // [T][K], or null (forward: 1)
  void* y;                   // [T][H] (forward)
  const void* dy;            // [T][H] (backward)
  void* drows;               // [T*K][H] or null
  float* dweights;           // [T][K] or null
  int64_t T, R, H;
  int E, K, element;
};
hipError_t launch_combine_tokens(const CombineTokensArgs& a, hipStream_t s);
hipError_t launch_combine_backward(const CombineTokensArgs& a, hipStream_t s);

// -------------------------------------------------------------- activation
struct SwigluArgs {
  const void* h;             // [M][2I]
  void* a;                   // [M][I]
  int8_t* q;                 // [M][2I] codes of h, or null
  float* s;                  // [M][2][ceil(I/128)]
  const void* da;            // [M][I] (backward)
  void* dh;                  // [M][2I] (backward)
  int64_t groups;            // M * ceil(I/128), below 2^31
  int I, element;
  int turn;                  // 0: gate columns, then up columns; else in turns of so many (a multiple of 8 that divides I)
  float clamp;               // +inf: none
};
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s);
hipError_t launch_swiglu_backward(const SwigluArgs& a, hipStream_t s);

// ------------------------------------------------- 8-bit integer product
struct Int8Args {
  const uint8_t* a;          // int8 [M][K]
  const float* as;           // [M]
  const void* x;             // [M][K] (quantised on the way), or null
  const uint8_t* b;          // int8 [G][N][K]
  const float* bs;           // [G][N]
  const int32_t* offsets;    // as in BlockArgs
  const int32_t* counts;
  void* y;                   // [M][N]
  int64_t M;
  int tail;                  // rows behind the M ones, streamed
  int N, K, G;
  int x_element, y_element;
};
hipError_t launch_int8_quantize(const void* x, int element, int64_t rows, int cols, uint8_t* q, float* s, hipStream_t st);
// whether launch_int8_gemm may quantise a.x on the way (a.a and a.as unused)
bool int8_from_x(const Int8Args& a);
hipError_t launch_int8_gemm(const Int8Args& a, int num_cus, hipStream_t s);

}  // namespace mm
