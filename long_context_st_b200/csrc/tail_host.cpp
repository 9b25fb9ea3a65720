// Host side of the tail cache: page layout, tree masks and rotary frequencies.
#include <cmath>

#include "pages.cuh"

namespace jolt {

bool pages_ok(const jolt_pages* p) {
  if (!p || p->n_pages < 1 || p->n_kv < 1 || p->n_kv > 4096) return false;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return false;
  if (p->d_h != 64 && p->d_h != 128) return false;
  if (p->b_k != 2 && p->b_k != 4 && p->b_k != 8) return false;
  if (p->b_v != 2 && p->b_v != 4 && p->b_v != 8) return false;
  return p->io_dtype == JOLT_F32 || p->io_dtype == JOLT_BF16;
}

}  // namespace jolt

using namespace jolt;

extern "C" {

jolt_status jolt_pages_layout(const jolt_pages* p, uint64_t offsets[4], uint64_t* page_bytes) {
  if (!pages_ok(p)) return JOLT_ERR_INVALID_ARG;
  const PageLayout l = page_layout(*p);
  if (offsets) {
    offsets[0] = l.kc;
    offsets[1] = l.ks;
    offsets[2] = l.vc;
    offsets[3] = l.vs;
  }
  if (page_bytes) *page_bytes = l.bytes;
  return JOLT_OK;
}

uint64_t jolt_pages_bytes(const jolt_pages* p) {
  return pages_ok(p) ? uint64_t(p->n_pages) * page_layout(*p).bytes : 0;
}

jolt_status jolt_tree_mask(const int32_t* parents, int32_t n, uint64_t* mask) {
  if (n < 0 || n > 64 || (n && (!parents || !mask))) return JOLT_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (parents[i] < -1 || parents[i] >= i) return JOLT_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) mask[i] = (parents[i] < 0 ? 0 : mask[parents[i]]) | (uint64_t(1) << i);
  return JOLT_OK;
}

jolt_status jolt_rope_freqs(int32_t rot_dim, double theta, int32_t mode, double factor, int32_t original_len,
                            double low, double high, float* inv_freq, float* scaling_out) {
  if (rot_dim < 2 || rot_dim > 512 || rot_dim % 2 || !(theta > 0.0) || !std::isfinite(theta) || !inv_freq)
    return JOLT_ERR_INVALID_ARG;
  if (mode < JOLT_ROPE_PLAIN || mode > JOLT_ROPE_YARN) return JOLT_ERR_INVALID_ARG;
  if (mode != JOLT_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return JOLT_ERR_INVALID_ARG;
  if (mode == JOLT_ROPE_NTK && rot_dim < 4) return JOLT_ERR_INVALID_ARG;
  const bool ramp = mode == JOLT_ROPE_RAMP || mode == JOLT_ROPE_YARN;
  if (ramp && (original_len < 1 || !(low > 0.0) || !(low < high) || !std::isfinite(high))) return JOLT_ERR_INVALID_ARG;
  if (mode == JOLT_ROPE_YARN && !(theta > 1.0)) return JOLT_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  if (mode == JOLT_ROPE_NTK) theta *= std::pow(factor, double(rot_dim) / (rot_dim - 2));
  // pair index whose pair turns `turns` times over original_len tokens: original_len * f_i = 2 pi turns
  auto index_of = [&](double turns) {
    return rot_dim * std::log(original_len / (two_pi * turns)) / (2.0 * std::log(theta));
  };
  double first = 0.0, last = 0.0;
  if (mode == JOLT_ROPE_YARN) {
    first = std::fmax(std::floor(index_of(high)), 0.0);
    last = std::fmin(std::ceil(index_of(low)), rot_dim - 1.0);
    if (last <= first) last = first + 1e-3;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(theta, -2.0 * i / rot_dim);
    double keep = 1.0;  // weight of the unscaled frequency
    if (mode == JOLT_ROPE_LINEAR) keep = 0.0;
    if (mode == JOLT_ROPE_RAMP) keep = (original_len * f / two_pi - low) / (high - low);
    if (mode == JOLT_ROPE_YARN) keep = 1.0 - (i - first) / (last - first);
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    inv_freq[i] = float(keep == 1.0 ? f : (1.0 - keep) * f / factor + keep * f);
  }
  if (scaling_out) *scaling_out = mode == JOLT_ROPE_YARN ? float(0.1 * std::log(factor) + 1.0) : 1.f;
  return JOLT_OK;
}

}  // extern "C"
