// Activations to 8 bits, with a power-of-two scale for every 32 columns of a
// row, and back; and their C calls.  The form itself: zero_rows.cuh.
//
// Memory is the floor of both: four lanes share a group, its largest magnitude takes
// two shuffles, and four rows are on their way to a thread.  32768 x 8192
// bf16 to e4m3 and back: 274 us of device time, 5.9 TB/s of the 1.63 GB read and
// written (whole numbers: 287).  Rows that
// are not 16-byte aligned are read as single elements and turned in shared
// memory before they are written: 4099 x 777 fp32, 11.5 us for both, of which the
// floor is 4.8.

#include "zero_flatstep.h"
#include "zero_rows.cuh"
#include "zero_rows_host.h"

namespace zfs {
namespace {

constexpr int kPackThreads = 256;
constexpr int kPackCtas = 5;  // of an SM (48 registers)

struct PackArgs {
  long long rows;
  int cols, lanes;     // lanes: threads on a row, a power of two up to kPackThreads
  int groups, form;
  void* x;             // read by the one, written by the other
  long long x_stride;
  uint8_t *codes, *scales;
};

// A thread takes eight columns of kRows rows at a time, `lanes` threads a row.
// kAligned: whole 16-byte words, else a warp's lanes all hold one row.
template <bool kFp32, bool kAligned, bool kPack, int kForm>
__global__ void __launch_bounds__(kPackThreads, kPackCtas) pack_kernel(const __grid_constant__ PackArgs a) {
  constexpr int kRows = kAligned ? 4 : kPack ? 2 : 1;  // in flight
  constexpr long long kSize = kFp32 ? 4 : 2;
  __shared__ __align__(16) float turned[kAligned || kPack ? 1 : kPackThreads / 32][256];
  const int lanes = a.lanes, lane = threadIdx.x % lanes, per_cta = kPackThreads / lanes;
  const long long step = static_cast<long long>(gridDim.x) * per_cta;
  const long long first = static_cast<long long>(blockIdx.x) * per_cta;
  for (long long r0 = first; r0 < a.rows; r0 += step * kRows) {
    const long long mine = r0 + threadIdx.x / lanes;
    for (int at = 0; at < a.cols; at += lanes * 8) {
      const int cols = a.cols - at, groups = a.groups - at / kPackGroup;
      Eight<kFp32, 8> raw[kRows];
      EightCodes codes[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const long long r = mine + step * i;
        const bool real = r < a.rows;
        if constexpr (kPack) {
          const char* row = static_cast<const char*>(a.x) + (r * a.x_stride + at) * kSize;
          if constexpr (kAligned) load_eight<kFp32, 8>(row, lane, lanes, real ? cols : 0, &raw[i]);
          else load_neighbours<kFp32>(row, lane, real ? cols : 0, &raw[i]);
        } else {
          load_codes(a.codes + r * a.groups * kPackGroup + at, a.scales + r * a.groups + at / kPackGroup, lane,
                     real ? groups : 0, &codes[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const long long r = mine + step * i;
        F2 x[4];
        if constexpr (kPack) {
          widen_pairs<kFp32, 8>(raw[i], x);
          pack_eight(x, lane, lanes, groups, r < a.rows, kForm, a.codes + r * a.groups * kPackGroup + at,
                     a.scales + r * a.groups + at / kPackGroup);
        } else {
          widen_codes(codes[i], kForm, x);
          char* row = static_cast<char*>(a.x) + (r * a.x_stride + at) * kSize;
          const bool real = r < a.rows;
          if constexpr (kAligned) {
            if (real) store_pairs<kFp32, 8>(row, lane, lanes, cols, x);
          } else {
            const int skip = lane / 32 * 256;  // the same row for the whole warp
            store_neighbours<kFp32>(row + skip * kSize, real ? cols - skip : 0, x, turned[threadIdx.x / 32]);
          }
        }
      }
    }
  }
}

template <bool kPack, int kForm>
void launch_pack(const PackArgs& a, bool fp32, bool aligned, int ctas, cudaStream_t s) {
  if (fp32) {
    if (aligned) pack_kernel<true, true, kPack, kForm><<<ctas, kPackThreads, 0, s>>>(a);
    else pack_kernel<true, false, kPack, kForm><<<ctas, kPackThreads, 0, s>>>(a);
  } else {
    if (aligned) pack_kernel<false, true, kPack, kForm><<<ctas, kPackThreads, 0, s>>>(a);
    else pack_kernel<false, false, kPack, kForm><<<ctas, kPackThreads, 0, s>>>(a);
  }
}

zero_status convert(int64_t rows, int64_t cols, const void* x, int32_t dtype, int64_t x_stride,
                    const zero_packed* packed, bool pack, void* stream) {
  if (rows < 0) return refuse(ZERO_EINVAL, "rows is negative");
  if (cols < 1 || cols > (1 << 24)) return refuse(ZERO_EINVAL, "cols not in 1..2^24");
  if (!is_dtype(dtype)) return refuse(ZERO_EINVAL, "dtype is neither bf16 (0) nor fp32 (1)");
  if (!packed) return refuse(ZERO_EINVAL, "packed is NULL");
  if (packed->format != ZERO_PACK_E4M3 && packed->format != ZERO_PACK_INT8)
    return refuse(ZERO_EINVAL, "the 8-bit format is neither e4m3 (0) nor int8 (1)");
  if (rows == 0) return ZERO_OK;
  if (misplaced(x, dtype_bytes(dtype)) || x_stride < 0)
    return refuse(ZERO_EINVAL, "the matrix is NULL or misaligned, or its stride negative");
  if (!pack && rows_overlap(x_stride, rows, cols)) return refuse(ZERO_EINVAL, "out's stride makes its rows overlap");
  if (misplaced(packed->codes, 16) || !packed->scales)
    return refuse(ZERO_EINVAL, "codes or scales are NULL or misaligned");
  PackArgs a{};
  a.rows = rows;
  a.cols = static_cast<int>(cols);
  a.groups = (a.cols + kPackGroup - 1) / kPackGroup;
  a.form = packed->format == ZERO_PACK_E4M3 ? kPackE4m3 : kPackInt8;
  a.x = const_cast<void*>(x);
  a.x_stride = x_stride;
  a.codes = static_cast<uint8_t*>(packed->codes);
  a.scales = static_cast<uint8_t*>(packed->scales);
  const bool aligned = cols % 8 == 0 && rows_aligned(x, x_stride, rows, dtype);
  const int need = (a.cols + 7) / 8, lanes = power_of_two(need < kPackThreads ? need : kPackThreads);
  a.lanes = aligned || lanes >= 32 ? lanes : 32;
  const long long per_cta = kPackThreads / a.lanes, want = (rows + per_cta - 1) / per_cta;
  const long long most = static_cast<long long>(sm_count()) * kPackCtas;
  const int ctas = static_cast<int>(want < most ? want : most);
  const bool fp32 = dtype == ZERO_GRAD_FP32, e4m3 = a.form == kPackE4m3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pack) e4m3 ? launch_pack<true, kPackE4m3>(a, fp32, aligned, ctas, s) : launch_pack<true, kPackInt8>(a, fp32, aligned, ctas, s);
  else e4m3 ? launch_pack<false, kPackE4m3>(a, fp32, aligned, ctas, s) : launch_pack<false, kPackInt8>(a, fp32, aligned, ctas, s);
  return launch_status(pack ? "pack launch" : "unpack launch");
}

}  // namespace

}  // namespace zfs

extern "C" {

zero_status zero_pack_activations(int64_t rows, int64_t cols, const void* x, int32_t dtype, int64_t x_stride,
                                  const zero_packed* packed, void* stream) {
  return zfs::convert(rows, cols, x, dtype, x_stride, packed, true, stream);
}

zero_status zero_unpack_activations(int64_t rows, int64_t cols, const zero_packed* packed, void* out, int32_t dtype,
                                    int64_t out_stride, void* stream) {
  return zfs::convert(rows, cols, out, dtype, out_stride, packed, false, stream);
}

}  // extern "C"
