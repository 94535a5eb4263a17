// C-ABI entry points of moe_experts.h: host-side argument checks, then kernel
// launches on the caller's stream. Nothing here allocates, frees or
// synchronises.
#include "experts.hpp"

#include <atomic>
#include <cmath>
#include <cstring>

#include "moe_experts.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace moe;

static_assert(MOE_GATE_BF16 == kGateBf16 && MOE_GATE_SIGMOID == kGateSigmoid &&
                  MOE_GATE_RENORM == kGateRenorm && MOE_STATUS_BAD_LOGIT == kStBadLogit &&
                  MOE_STATUS_BAD_SLOT == kStBadSlot && MOE_STATUS_BAD_EXPERT == kStBadExpert &&
                  MOE_FP8_ROUND_SCALE == kFp8RoundScale && MOE_FP8_UE8M0 == kFp8Ue8m0 &&
                  MOE_FP8_SCALE_ROWS == kFp8ScaleRows,
              "flags or status bits of the header and the kernels differ");

constexpr int kDevices = 64;
std::atomic<int> g_device_arch[kDevices];  // 0 = not checked yet, 1 = gfx950, 2 = other

// The kernels are compiled for gfx950 only; refuse any other current device.
int current_device_ok() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MOE_ERR_DEVICE;
  int state = dev < kDevices ? g_device_arch[dev].load(std::memory_order_relaxed) : 0;
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOE_ERR_DEVICE;
    state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    if (dev < kDevices) g_device_arch[dev].store(state, std::memory_order_relaxed);
  }
  return state == 1 ? MOE_OK : MOE_ERR_ARCH;
}

bool on(const void *p, uintptr_t bytes) {  // aligned to that many bytes (a power of two)
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

// A launch holds fewer than 2^32 threads: at most this many waves, with a
// workgroup to spare.
constexpr int64_t kMaxWaveRows = (1 << 26) - 64;

// The FP8 flags and the channel counts they need.
int fp8_flags_ok(int32_t channels, int32_t flags) {
  constexpr int kCast = MOE_FP8_ROUND_SCALE | MOE_FP8_UE8M0;
  if (flags & ~(kCast | MOE_FP8_SCALE_ROWS)) return MOE_ERR_FLAGS;
  if ((flags & kCast) == MOE_FP8_UE8M0) return MOE_ERR_FLAGS;  // needs power-of-two scales
  if (channels % (flags & MOE_FP8_UE8M0 ? 4 * kFp8Group : kFp8Group)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int gate_ok(int32_t T, int32_t E, int32_t K, int32_t flags, float scale) {
  if (T < 0 || E < 1 || E > kMaxExperts || K < 1 || K > 64 || K > E) return MOE_ERR_SHAPE;
  if (T > kMaxWaveRows) return MOE_ERR_SHAPE;
  if (flags & ~(MOE_GATE_BF16 | MOE_GATE_SIGMOID | MOE_GATE_RENORM)) return MOE_ERR_FLAGS;
  if (!std::isfinite(scale)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int segments_ok(int32_t E, int64_t rows) {
  if (E < 1 || E > kMaxExperts || rows < 0 || rows >= ((int64_t)1 << 31)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

}  // namespace

MOE_API int moe_gate(int32_t T, int32_t E, int32_t K, const void *logits, int64_t *topk_idx,
                     float *topk_weights, int32_t flags, float scale, int32_t *status,
                     hipStream_t stream) {
  int rc = gate_ok(T, E, K, flags, scale);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_weights) return MOE_ERR_NULL;
  if (!on(logits, flags & MOE_GATE_BF16 ? 2 : 4) || !on(topk_idx, 8) || !on(topk_weights, 4))
    return MOE_ERR_ALIGN;
  rc = current_device_ok();
  if (rc) return rc;
  return launched(launch_gate(logits, T, E, K, flags, scale, topk_idx, topk_weights, status,
                              stream));
}

MOE_API int moe_gate_grad(int32_t T, int32_t E, int32_t K, const void *logits,
                          const int64_t *topk_idx, const float *d_weights, void *d_logits,
                          int32_t flags, float scale, int32_t *status, hipStream_t stream) {
  int rc = gate_ok(T, E, K, flags, scale);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !d_weights || !d_logits) return MOE_ERR_NULL;
  const uintptr_t el = flags & MOE_GATE_BF16 ? 2 : 4;
  if (!on(logits, el) || !on(d_logits, el) || !on(topk_idx, 8) || !on(d_weights, 4))
    return MOE_ERR_ALIGN;
  rc = current_device_ok();
  if (rc) return rc;
  return launched(launch_gate_grad(logits, topk_idx, d_weights, T, E, K, flags, scale, d_logits,
                                   status, stream));
}

MOE_API int moe_combine_grad(const moe_shape *s, const uint16_t *d_out, const uint16_t *y,
                             int64_t recv_rows, const int32_t *slot, const float *topk_weights,
                             uint16_t *d_y, float *d_weights, const int64_t *topk_idx,
                             const int32_t *rank_mask, int32_t *status, hipStream_t stream) {
  if (!s) return MOE_ERR_NULL;
  if (s->T < 0 || s->K < 1 || s->K > 64 || s->E < 1 || s->E > kMaxExperts || s->R < 1 ||
      s->E % s->R != 0 || s->A < 1 || s->A > (1 << 16) || s->H < 8 || s->H > (1 << 20) ||
      s->H % 8 != 0)
    return MOE_ERR_SHAPE;
  // one workgroup of four waves per pair, tokens rounded up to eights
  if (((int64_t)s->T + 7) * s->K * 4 > kMaxWaveRows) return MOE_ERR_SHAPE;
  if (recv_rows < 0) return MOE_ERR_CAPACITY;
  if (!topk_idx != !rank_mask) return MOE_ERR_NULL;
  if (s->T == 0) return MOE_OK;
  if (!d_out || !slot || (recv_rows > 0 && (!d_y || (d_weights && !y)))) return MOE_ERR_NULL;
  if (!on(d_out, 16) || !on(y, 16) || !on(d_y, 16) || !on(topk_idx, 8) || !on(slot, 4) ||
      !on(topk_weights, 4) || !on(d_weights, 4))
    return MOE_ERR_ALIGN;
  int rc = current_device_ok();
  if (rc) return rc;
  const uint64_t L = (uint64_t)(s->E / s->R);
  const CombineMask cm{topk_idx, rank_mask, s->E, ((1ull << 32) + L - 1) / L};
  return launched(launch_combine_grad(d_out, y, recv_rows, slot, topk_weights, d_y, d_weights,
                                      s->T, s->K, s->H, cm, status, stream));
}

MOE_API int moe_grouped_gemm_fp8(int32_t E, int32_t N, int32_t C, const uint8_t *a,
                                 const void *a_scale, int64_t rows, const int32_t *row_start,
                                 const int32_t *count, const uint8_t *w, const float *w_scale,
                                 uint16_t *out, int32_t flags, int32_t max_count, int32_t *status,
                                 hipStream_t stream) {
  int rc = segments_ok(E, rows);
  if (rc) return rc;
  if (N < 8 || N > (1 << 20) || N % 8 != 0 || C < kFp8Group || C > (1 << 20) || max_count < 0)
    return MOE_ERR_SHAPE;
  rc = fp8_flags_ok(C, flags);
  if (rc) return rc;
  const bool columns = !(flags & MOE_FP8_SCALE_ROWS);
  if (columns && rows % E != 0) return MOE_ERR_SHAPE;
  if (!row_start || !count) return MOE_ERR_NULL;
  if (rows == 0) return MOE_OK;
  if (!a || !a_scale || !w || !w_scale || !out) return MOE_ERR_NULL;
  if (!on(a, 16) || !on(w, 16) || !on(out, 16) || !on(a_scale, 4) || !on(w_scale, 4) ||
      !on(row_start, 4) || !on(count, 4))
    return MOE_ERR_ALIGN;
  rc = current_device_ok();
  if (rc) return rc;
  const Segments seg{row_start, count, E, rows, columns ? (int32_t)(rows / E) : 0, max_count,
                     0, 0};
  const GemmArgs g{a, a_scale, w, w_scale, out, N, C, flags, status};
  return launched(launch_grouped_gemm(seg, g, stream));
}

MOE_API int moe_swiglu_fp8(int32_t E, int32_t I, int64_t rows, const uint16_t *x,
                           const int32_t *row_start, const int32_t *count, uint8_t *q,
                           void *scale, int32_t flags, int32_t *status, hipStream_t stream) {
  int rc = segments_ok(E, rows);
  if (rc) return rc;
  if (I < kFp8Group || I > (1 << 20)) return MOE_ERR_SHAPE;
  rc = fp8_flags_ok(I, flags);
  if (rc) return rc;
  if (!row_start || !count) return MOE_ERR_NULL;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_NULL;
  if (!on(x, 16) || !on(q, 16) || !on(scale, 4) || !on(row_start, 4) || !on(count, 4))
    return MOE_ERR_ALIGN;
  rc = current_device_ok();
  if (rc) return rc;
  const Segments seg{row_start, count, E, rows, 0, 0, 0, 0};
  return launched(launch_swiglu_fp8(seg, I, x, q, scale, flags, status, stream));
}

MOE_API int moe_swiglu_grad(int32_t E, int32_t I, int64_t rows, const uint16_t *x,
                            const uint16_t *d_h, const int32_t *row_start, const int32_t *count,
                            uint16_t *d_x, int32_t *status, hipStream_t stream) {
  int rc = segments_ok(E, rows);
  if (rc) return rc;
  if (I < 8 || I > (1 << 20) || I % 8 != 0) return MOE_ERR_SHAPE;
  if (!row_start || !count) return MOE_ERR_NULL;
  if (rows == 0) return MOE_OK;
  if (!x || !d_h || !d_x) return MOE_ERR_NULL;
  if (!on(x, 16) || !on(d_h, 16) || !on(d_x, 16) || !on(row_start, 4) || !on(count, 4))
    return MOE_ERR_ALIGN;
  rc = current_device_ok();
  if (rc) return rc;
  const Segments seg{row_start, count, E, rows, 0, 0, 0, 0};
  return launched(launch_swiglu_grad(seg, I, x, d_h, d_x, status, stream));
}
