// Arguments and workspace of the low-rank adapters' operators, and of the balance loss and the
// gradient of the routing.
#pragma once

#include "fp8_internal.h"

namespace bl {

// The rows of a call, their adapters, and the values that an adapter's pass goes through. A pass
// works on one of the two weights, w [L, R, D]: a with D = K or b with D = N.
struct AdapterRows {
  const int32_t* index;  // [M]
  int64_t M, L, R;
};

struct AdapterForwardArgs {
  AdapterRows rows;
  const void* x;         // [M, K], rows ldx elements apart
  int64_t K, ldx;
  const void* a;         // [L, R, K]
  const void* b;         // [L, R, N]
  int dtype;             // of x, a and b
  int64_t N;
  const float* scale;    // [L] or null
  const void* base;      // [M, N] or null
  int64_t ldbase;
  void* y;               // [M, N]
  int ydtype;            // of base and y
  int64_t ldy;
  float* h;              // [M, R]
};

struct AdapterBackwardArgs {
  AdapterRows rows;
  const void* x;         // [M, K], rows ldx elements apart
  int64_t K, ldx;
  const void* a;         // [L, R, K]
  const void* b;         // [L, R, N]
  int dtype;             // of x, a and b
  int64_t N;
  const float* scale;    // [L] or null
  const float* h;        // [M, R]
  const void* dy;        // [M, N]
  int dydtype;
  int64_t lddy;
  const void* base;      // [M, K] or null
  int64_t ldbase;
  void* dx;              // [M, K] or null
  int dxdtype;           // of base and dx
  int64_t lddx;
  float* da;             // [L, R, K]
  float* db;             // [L, R, N]
  int add;               // onto what da and db hold
};

// Scratch of one call: the rows sorted by adapter, and what passes hand on. 256-byte aligned
// regions, no fill needed; nothing at all for few rows (forward).
struct AdapterWs {
  size_t order_off;      // int32 [rows] row of each sorted place, -1 for none
  size_t tile_off;       // int32 [tiles] adapter of each tile, L for rows without one
  size_t start_off;      // int32 [L + 2] first tile of each adapter, of the rows without one, and the end
  size_t count_off;      // int32 [chunks, L + 1], more than one chunk of the sort
  size_t arrived_off;    // uint32 [counters] workgroups that have ended, cleared by the sort
  int64_t counters;
  size_t part_off;       // fp32 [splits, rows, RP] partial sums of the products over K or N
  size_t c_off[3];       // the scaled h (forward) or dh, sorted, in each layout that is needed
  size_t hc_off[3];      // the scaled h (backward)
  size_t sum_off[2];     // fp32 [2 shares, R, D] partial sums over rows, of da and of db (backward)
  size_t total;
};
AdapterWs adapter_ws(int64_t M, int64_t L, int64_t R, int64_t K, int64_t N, bool backward);

hipError_t launch_adapter_forward(const AdapterForwardArgs& a, char* ws, hipStream_t s);
hipError_t launch_adapter_backward(const AdapterBackwardArgs& a, char* ws, hipStream_t s);

// What the balance loss and the routing's gradient know of the rows.
struct RouteRows {
  const void* logits;    // [M, E], rows ld elements apart
  int dtype;
  int64_t M, E, ld;
  const int32_t* index;  // [M, k]
  int k;
  int sigmoid;           // else softmax
  const int32_t* offsets;  // [S + 1] or null: all rows are one sequence
  int64_t S;
};
struct RouteBalanceArgs {
  RouteRows r;
  float* loss;           // [S]
  int32_t* count;        // [S, E]
  float* coef;           // [S, E]
};
struct RouteBackwardArgs {
  RouteRows r;
  const float* dweight;  // [M, k] or null
  int renorm;
  float factor;
  const float* coef;     // [S, E] or null
  const float* dloss;    // [S], with coef
  void* dlogits;         // [M, E], rows ldd elements apart
  int ddtype;
  int64_t ldd;
};
size_t route_balance_ws_bytes(int64_t M, int64_t E, int64_t S);
hipError_t launch_route_balance(const RouteBalanceArgs& a, char* ws, hipStream_t s);
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s);

}  // namespace bl
