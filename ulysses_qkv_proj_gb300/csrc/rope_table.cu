// rope_table.cu -- the cos/sin table that the norm and projection calls read, for plain and scaled rotary positions.
//
//   row p = m [cos(p f_0) .. cos(p f_{h-1}) | sin(p f_0) .. sin(p f_{h-1})],  h = rot / 2
//
// The h frequencies are formed once on the host in 64 bits and passed as fractions of a turn, rounded to units of 2^-64.  A phase
// is then one integer product modulo 2^64: the multiples of a turn fall off exactly, so that position p adds at most p 2^-65 of a
// turn (2^-34 at the last one) to what the 64-bit rounding of its frequency is, and no angle is ever reduced in floating
// point.  The quarter turn is taken off the integer too, and the rest, in [-1/8, 1/8] turn, becomes a float that
// keeps its leading bits however small it is.  Sine and cosine of it are
// polynomials of odd and even powers, fitted for the least relative error by weighted least squares (4e-9 and
// 6e-11 before rounding; evaluated in fp32 at most 0.8 and 1.0 units in the last place off, 0.3 on average).
//
// Bound: HBM writes: 524288 positions of 512 bytes take 44.2 us, 6.1 TB/s.  A thread forms four pairs of a row and writes two
// 16-byte pieces, and goes on to the same pairs of three more rows, so that the frequencies are loaded once for four (with sincospif
// and a row a thread it was bound by instructions and took 129 us).
#include "../../include/qnre.h"
#include "api_util.cuh"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace {

using namespace qnre;
using namespace qnre::api;

constexpr int kMaxPairs = QNRE_HEAD_DIM / 2;
constexpr int kThreads = 256;

struct TableArgs {
  float* out;
  long long first;
  uint32_t n_pos, quads, rows;  // quads: groups of four pairs in a row; rows: of a thread
  float magnitude;
  uint64_t turn[kMaxPairs];  // a position's share of a turn, 2^-64
};

__device__ __forceinline__ void cos_sin_of(uint64_t phase, float& c, float& s) {
  const uint64_t nearest = phase + (1ull << 61);  // its top two bits: the nearest quarter turn
  const uint32_t top = static_cast<uint32_t>(nearest >> 32), low = static_cast<uint32_t>(nearest);
  const int rest = static_cast<int>(top & 0x3FFFFFFFu) - (1 << 29);  // 2^-32 of a turn, and 23 bits behind them
  const float behind = __uint_as_float(0x3F800000u | low >> 9) - 1.f;
  const float h = (static_cast<float>(rest) + behind) * 4.656612873077393e-10f;  // half turns: 2^-31
  const float z = h * h;
  const float odd = fmaf(z, fmaf(z, fmaf(z, -0.5894187688827515f, 2.549805164337158f), -5.167708873748779f),
                         -8.742277657347586e-08f);  // the rest of pi behind 3.14159274
  const float sn = fmaf(h, 3.1415927410125732f, h * odd);
  const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 0.23136422038078308f, -1.3350505828857422f), 4.0587077140808105f),
                                -4.934802055358887f), 1.f);
  const uint32_t quarter = top >> 30;
  const float x = quarter & 1 ? sn : cs, y = quarter & 1 ? cs : sn;
  c = __uint_as_float(__float_as_uint(x) ^ ((quarter + 1) << 30 & 0x80000000u));
  s = __uint_as_float(__float_as_uint(y) ^ (quarter << 30 & 0x80000000u));
}

__global__ void __launch_bounds__(kThreads) table_kernel(const __grid_constant__ TableArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t per = kThreads / a.quads, sub = threadIdx.x / a.quads, quad = threadIdx.x - sub * a.quads;
  if (sub >= per) return;
  uint64_t turn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) turn[i] = a.turn[quad * 4 + i];
  uint32_t row = blockIdx.x * per * a.rows + sub;
  for (uint32_t k = 0; k < a.rows && row < a.n_pos; ++k, row += per) {
    const uint64_t p = static_cast<uint64_t>(a.first + row);
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cos_sin_of(p * turn[i], c[i], s[i]);
      c[i] *= a.magnitude;
      s[i] *= a.magnitude;
    }
    float4* dst = reinterpret_cast<float4*>(a.out) + static_cast<uint64_t>(row) * (2 * a.quads) + quad;
    dst[0] = make_float4(c[0], c[1], c[2], c[3]);
    dst[a.quads] = make_float4(s[0], s[1], s[2], s[3]);
  }
}

}  // namespace

extern "C" qnre_status_t qnre_rope_table(float* cos_sin, int64_t n_pos, int rot, int64_t first, double theta,
                                         const qnre_rope_scaling_t* scaling, qnre_stream_t stream) {
  qnre_rope_scaling_t s{QNRE_ROPE_SCALE_NONE, 1.0, 0.0, 0.0, 0.0, 1.0};
  if (scaling != nullptr) s = *scaling;
  if (n_pos < 0 || first < 0 || rot < 1 || rot % 16 != 0 || !(theta > 1.0) || !std::isfinite(theta) ||
      !std::isfinite(static_cast<float>(s.magnitude)))
    return QNRE_ERR_INVALID_ARG;
  const bool ramp = s.kind == QNRE_ROPE_SCALE_YARN || s.kind == QNRE_ROPE_SCALE_WAVELENGTH;
  if (s.kind < QNRE_ROPE_SCALE_NONE || s.kind > QNRE_ROPE_SCALE_WAVELENGTH) return QNRE_ERR_INVALID_ARG;
  if (s.kind != QNRE_ROPE_SCALE_NONE && !(s.factor > 0.0 && std::isfinite(s.factor))) return QNRE_ERR_INVALID_ARG;
  if (ramp && !(s.original > 0.0 && std::isfinite(s.original) && s.low > 0.0 && s.high > s.low && std::isfinite(s.high)))
    return QNRE_ERR_INVALID_ARG;
  if (rot > QNRE_HEAD_DIM) return QNRE_ERR_UNSUPPORTED;
  if (n_pos > (int64_t{1} << 31) || first > (int64_t{1} << 31) - n_pos) return QNRE_ERR_CAPACITY;
  if (n_pos == 0) return QNRE_OK;
  if (cos_sin == nullptr) return QNRE_ERR_INVALID_ARG;
  if (!aligned(cos_sin, 16)) return QNRE_ERR_ALIGNMENT;

  TableArgs a{};
  a.out = cos_sin;
  a.n_pos = static_cast<uint32_t>(n_pos);
  a.first = first;
  a.quads = rot / 8;
  a.magnitude = static_cast<float>(s.magnitude);
  const double two_pi = 6.283185307179586476925;
  const double base = s.kind == QNRE_ROPE_SCALE_BASE ? theta * std::pow(s.factor, rot / (rot - 2.0)) : theta;
  if (!(base > 0.0) || !std::isfinite(base)) return QNRE_ERR_INVALID_ARG;
  // the (fractional) pair that makes so many turns over the original length
  auto pair_of = [&](double turns) { return rot * std::log(s.original / (turns * two_pi)) / (2.0 * std::log(theta)); };
  double lo = 0.0, hi = 0.0;
  if (s.kind == QNRE_ROPE_SCALE_YARN) {
    lo = std::max(std::floor(pair_of(s.high)), 0.0);
    hi = std::min(std::ceil(pair_of(s.low)), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (s.kind == QNRE_ROPE_SCALE_LINEAR) {
      f /= s.factor;
    } else if (s.kind == QNRE_ROPE_SCALE_YARN) {
      const double slow = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      f = f * (slow / s.factor + (1.0 - slow));
    } else if (s.kind == QNRE_ROPE_SCALE_WAVELENGTH) {
      const double keep = std::min(std::max((s.original * f / two_pi - s.low) / (s.high - s.low), 0.0), 1.0);
      f = f * (keep + (1.0 - keep) / s.factor);
    }
    if (!std::isfinite(f)) return QNRE_ERR_INVALID_ARG;  // (a factor so small that a quotient leaves the range)
    const double turns = f / two_pi;  // a whole turn a position changes nothing
    a.turn[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(turns - std::floor(turns), 64)));
  }
  const int64_t per = kThreads / a.quads;
  a.rows = n_pos >= per * 152 * 64 ? 4 : 1;  // few rows: as many threads as there are
  const int64_t blocks = (n_pos + per * a.rows - 1) / (per * a.rows);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return from_cuda(cudaLaunchKernelEx(&cfg, table_kernel, a));
}
