// rope_table.cu -- the cos/sin table that the norm and projection calls read, for plain and scaled rotary positions.
//
//   row p = m [cos(p f_0) .. cos(p f_{h-1}) | sin(p f_0) .. sin(p f_{h-1})],  h = rot / 2
//
// The h frequencies are formed once on the host in 64 bits and passed as fractions of a turn in units of 2^-64.  A phase
// is then one integer product modulo 2^64: the multiples of a turn fall off exactly, so position 2^31 keeps the 2^-53 of its
// frequency and no angle is ever reduced in floating point.  The quarter turn is taken off the integer too, and the rest, in
// [-1/8, 1/8] turn, becomes a float that keeps its leading bits however small it is.
//
// Bound: the bytes written (a thread forms four pairs and writes two 16-byte pieces).
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
  long long n_pos, first;
  int quads;  // groups of four pairs in a row
  float magnitude;
  uint64_t turn[kMaxPairs];  // a position's share of a turn, 2^-64
};

__global__ void __launch_bounds__(kThreads) table_kernel(const __grid_constant__ TableArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long at = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long row = at / a.quads;
  if (row >= a.n_pos) return;
  const int quad = static_cast<int>(at - row * a.quads);
  const uint64_t p = static_cast<uint64_t>(a.first + row);
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t phase = p * a.turn[quad * 4 + i];
    const uint64_t nearest = phase + (1ull << 61);  // its top two bits: the nearest quarter turn
    const long long rest = static_cast<long long>((nearest & ~(3ull << 62)) - (1ull << 61));
    const float half_turns = fmaf(static_cast<float>(static_cast<int>(rest >> 32)), 4294967296.f,
                                  static_cast<float>(static_cast<uint32_t>(rest))) *
                             1.0842021724855044e-19f;  // 2^-63
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    const uint32_t quarter = static_cast<uint32_t>(nearest >> 62);
    const float x = (quarter & 1) ? sn : cs, y = (quarter & 1) ? cs : sn;
    c[i] = a.magnitude * (quarter == 1 || quarter == 2 ? -x : x);
    s[i] = a.magnitude * (quarter >= 2 ? -y : y);
  }
  float4* dst = reinterpret_cast<float4*>(a.out) + row * (2 * a.quads) + quad;
  dst[0] = make_float4(c[0], c[1], c[2], c[3]);
  dst[a.quads] = make_float4(s[0], s[1], s[2], s[3]);
}

}  // namespace

extern "C" qnre_status_t qnre_rope_table(float* cos_sin, int64_t n_pos, int rot, int64_t first, double theta,
                                         const qnre_rope_scaling_t* scaling, qnre_stream_t stream) {
  qnre_rope_scaling_t s{QNRE_ROPE_SCALE_NONE, 1.0, 0.0, 0.0, 0.0, 1.0};
  if (scaling != nullptr) s = *scaling;
  if (n_pos < 0 || first < 0 || rot < 1 || rot % 16 != 0 || !(theta > 1.0) || !std::isfinite(theta) ||
      !std::isfinite(s.magnitude))
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
  a.n_pos = n_pos;
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
    const double turns = f / two_pi;  // a whole turn a position changes nothing
    a.turn[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
  }
  const int64_t blocks = (n_pos * a.quads + kThreads - 1) / kThreads;
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
