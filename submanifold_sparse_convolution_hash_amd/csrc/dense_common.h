// What the dense layers' sources share on the host side and the small kernels
// around the tiled products (declared here, defined in linear.hip).
#pragma once

#include "submconv_internal.h"

namespace submconv {

// A 16-bit matrix of `rows` rows, `cols` columns, `ld` elements between rows;
// or `blocked` (dense_tile.h), then `cols` is a multiple of 64.
struct Mat16 {
  const uint16_t* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  bool blocked = false;
};
// A blocked matrix of the workspace and its bytes.
inline Mat16 blocked16(const void* p, int64_t rows, int64_t cols) {
  return Mat16{static_cast<const uint16_t*>(p), rows, cols, cols, true};
}
inline int64_t blocked_bytes(int64_t rows, int64_t cols) { return (rows + 127) / 128 * 128 * cols * 2; }


// Whether a product can read the matrix as it is: 16-byte pieces that start
// on 16 bytes and never straddle a row's end.
bool pieces_fit(const Mat16& a);

// A copy of a matrix whose column groups of `from_cols` are padded with zeros
// to `to_cols`, a multiple of 8.
struct PackJob {
  const uint16_t* from;
  int64_t rows, ld, from_cols, to_cols, row_pieces;
  uint16_t* to;
};
constexpr int kPacks = 4;
struct PackList {
  PackJob job[kPacks];
  int count = 0;
};
int run_packs(const PackList& list, hipStream_t stream);

// out[c] = sum over `parts` rows of partial[part][ld], c < cols, in order;
// columns of `groups` padded groups are closed up, and those from `split` on go
// to out2. Up to kSums of them in one launch.
struct SumJob {
  const float* partial;
  int64_t parts, ld, cols;
  int32_t groups;
  float* out;
  int64_t split = INT64_MAX;
  float* out2 = nullptr;
};
constexpr int kSums = 2;
struct SumList {
  SumJob job[kSums];
  int count = 0;
};
int run_sums(const SumList& list, hipStream_t stream);

// out[r][c] = sum over the `runs` planes [.. >= rows][ldp] of partial sums, in
// order, rounded once; columns of `groups` padded groups are closed up. Up to
// kPlanes of them in one launch.
struct PlaneJob {
  const float* partial;
  int64_t runs, plane, ldp, rows, cols;
  int32_t groups;
  uint16_t* out;
};
constexpr int kPlanes = 3;
struct PlaneList {
  PlaneJob job[kPlanes];
  int count = 0;
};
int run_planes(const PlaneList& list, bool bf16, hipStream_t stream);

// Column sums of a matrix in fp32 (bias gradients), with `partial` of
// column_parts(rows, cols) x round8(cols) floats; the last sum goes on the list.
int64_t column_parts(int64_t rows, int64_t cols);
int column_sums(const Mat16& a, bool bf16, float* partial, float* out, SumList* list,
                hipStream_t stream);

// dx[m][c] = sum_n dz[m][n] W[c][n] (both readable in pieces, or dz blocked),
// rounded once, dense. Small products are split over runs of n; `partial` of
// product_nt_bytes holds the runs' fp32 sums, whose addition goes on the list.
int64_t product_nt_bytes(int64_t rows, int64_t k, int64_t cols);
int product_nt(const Mat16& dz, const Mat16& W, bool bf16, float* partial, uint16_t* out,
               int64_t cols, PlaneList* list, hipStream_t stream);

// dW[c][n] = sum_m x[m][c] dz[m][n], rounded once; the rows are split over
// workgroups, `partial` of product_tn_bytes holds their fp32 sums, whose
// addition goes on the list. x and dz readable in pieces, one of them may be blocked; out is
// [cols_x][cols_z] dense, dz's columns in `groups` padded groups.
int64_t product_tn_bytes(int64_t rows, int64_t cin, int64_t cols);
int product_tn(const Mat16& x, const Mat16& dz, bool bf16, float* partial, uint16_t* out,
               int64_t cols_x, int64_t cols_z, int groups, PlaneList* list, hipStream_t stream);

// Linear layer: act(x W + bias) + residual, with operands readable in pieces,
// or x blocked.
int linear_forward(const Mat16& x, const Mat16& W, const float* bias, int act, bool bf16,
                   const uint16_t* residual, int64_t ldr, uint16_t* out, int64_t ldo, uint16_t* pre,
                   int64_t cols, hipStream_t stream);

// Forward products of 1 .. kFewRows rows, which read any matrix as it is
// (few_rows.hip): the linear layer, the gated block's hidden rows in fp32
// [rows][W_in.cols / 2], and its output from those.
constexpr int kFewRows = 8;
int few_linear(const Mat16& x, const Mat16& W, const float* bias, int act, bool bf16,
               const uint16_t* residual, int64_t ldr, uint16_t* out, uint16_t* pre,
               hipStream_t stream);
int few_gate(const Mat16& x, const Mat16& W, const float* bias, int act, bool bf16, float* h,
             uint16_t* pre, hipStream_t stream);
int few_out(const float* h, int64_t rows, const Mat16& W, const float* bias, bool bf16,
            const uint16_t* residual, int64_t ldr, uint16_t* out, hipStream_t stream);

// The gated block in one kernel, which keeps the hidden rows to itself
// (gated_fused.hip); operands readable in pieces, W_in in two groups.
bool fused_ffn_takes(int64_t rows, int64_t cin, int64_t hidden, int64_t cout);
int fused_ffn(const Mat16& x, const Mat16& W_in, int64_t F, const float* b_in, const Mat16& W_out,
              const float* b_out, int act, bool bf16, const uint16_t* residual, int64_t ldr,
              uint16_t* out, int64_t cout, hipStream_t stream);

// Cuts a caller's workspace into 256-byte aligned pieces, or, counting, only
// adds up what they take: the steps of an operator go through one function,
// which enqueues nothing while it counts.
struct Arena {
  bool counting = true;
  char* base = nullptr;
  int64_t used = 0;
  void* take(int64_t bytes) {
    void* p = counting ? nullptr : base + used;
    used += (bytes + 255) & ~int64_t{255};
    return p;
  }
};

// The matrix itself where products can read it in pieces and its column groups
// are multiples of `unit` (8; 64 where its columns are the k of a blocked
// matrix), else its padded copy in the arena, which is then on the list.
Mat16 readable(const Mat16& a, int groups, int unit, Arena& ws, PackList* list);

// Argument checks shared by the entry points.
int check_matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld);
int check_shape(const char* name, int64_t rows, int64_t cols);
int check_kind(int32_t act, int32_t dtype);
int check_workspace(const void* ws, int64_t have, int64_t need);

// A stand-in for a matrix in a workspace query: readable as it is, or not.
Mat16 shape_of(int64_t rows, int64_t cols, bool aligned);

#define SUBMCONV_TRY(expr)              \
  do {                                  \
    const int st_ = (expr);             \
    if (st_ != SUBMCONV_OK) return st_; \
  } while (0)

}  // namespace submconv
