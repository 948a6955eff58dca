// C ABI of the operators around the layer (dense packed projection, beam
// search's selection and reordering): host-side validation and dispatch.  No
// allocation, no host synchronisation, no state.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "moe.h"
#include "moe_internal.h"

namespace {

using namespace moe;

constexpr int kMaxCols = 65536;
constexpr int kMaxRows = 1 << 24;
constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxBeams = 64;
constexpr int kMaxOut = 128;
constexpr int kMaxVocab = 1 << 24;
constexpr int64_t kMaxBeamRows = 1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 40;  // any stride, count or size: products stay inside 64 bits

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool act_ok(int act) { return act == MOE_ACT_F32 || act == MOE_ACT_BF16; }
size_t act_size(int act) { return act == MOE_ACT_BF16 ? 2 : 4; }

moe_status dev(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_E_DEVICE; }

#define MOE_TRY(expr)                         \
  do {                                        \
    const moe_status st_ = (expr);            \
    if (st_ != MOE_OK) return st_;            \
  } while (0)

moe_status check_linear(const moe_linear* L) {
  if (!L) return MOE_E_ARG;
  if (L->rows < 1 || L->cols < 1 || L->cols % kGroup) return MOE_E_ARG;
  if (L->rows > kMaxRows || L->cols > kMaxCols) return MOE_E_UNSUPPORTED;
  if (L->qfmt != MOE_Q4_SYM_G32 && L->qfmt != MOE_Q2_ASYM_G32 && L->qfmt != MOE_Q3_SYM_G32) return MOE_E_UNSUPPORTED;
  if (!act_ok(L->act) || !act_ok(L->out)) return MOE_E_UNSUPPORTED;
  if (!L->w.codes || !L->w.scales || !aligned(L->w.codes, 16) || !aligned(L->w.scales, 2)) return MOE_E_ARG;
  if (L->qfmt == MOE_Q2_ASYM_G32 && (!L->w.mins || !aligned(L->w.mins, 2))) return MOE_E_ARG;
  if (L->bias && !aligned(L->bias, 4)) return MOE_E_ARG;
  return MOE_OK;
}

moe_status check_beam(const moe_beam* b) {
  if (!b) return MOE_E_ARG;
  if (b->batch < 0 || b->beams < 1 || b->vocab < 1 || b->n_out < 1) return MOE_E_ARG;
  if (b->eos < -1 || b->eos >= b->vocab) return MOE_E_ARG;
  if (b->beams > kMaxBeams || b->vocab > kMaxVocab || b->n_out > kMaxOut) return MOE_E_UNSUPPORTED;
  if ((int64_t)b->batch * b->beams > kMaxBeamRows) return MOE_E_UNSUPPORTED;
  if (!act_ok(b->act)) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

bool stride_ok(int64_t v) { return v >= 0 && v <= kMaxStride; }

// Bytes from the first to one past the last byte of a state's rows.
int64_t span(int64_t rows, int64_t row_stride, int64_t chunks, int64_t chunk_stride, int64_t bytes) {
  return (rows > 1 ? (rows - 1) * row_stride : 0) + (chunks > 1 ? (chunks - 1) * chunk_stride : 0) + bytes;
}

moe_status check_state(const moe_state& s, int64_t rows) {
  if (s.chunk_bytes < 0 || s.chunks < 0) return MOE_E_ARG;
  if (s.chunk_bytes == 0 || s.chunks == 0) return MOE_OK;
  if (!s.src || !s.dst) return MOE_E_ARG;
  if (s.chunk_bytes > kMaxStride || s.chunks > ((int64_t)1 << 22)) return MOE_E_UNSUPPORTED;
  if (rows > 1 && (!stride_ok(s.src_row_stride) || !stride_ok(s.dst_row_stride))) return MOE_E_ARG;
  if (s.chunks > 1 && (!stride_ok(s.src_chunk_stride) || !stride_ok(s.dst_chunk_stride))) return MOE_E_ARG;
  const int64_t sspan = span(rows, s.src_row_stride, s.chunks, s.src_chunk_stride, s.chunk_bytes);
  const int64_t dspan = span(rows, s.dst_row_stride, s.chunks, s.dst_chunk_stride, s.chunk_bytes);
  // written pieces lie apart: whole rows one after the other, or whole columns of pieces
  const int64_t row_span = span(1, 0, s.chunks, s.dst_chunk_stride, s.chunk_bytes);
  const int64_t col_span = span(rows, s.dst_row_stride, 1, 0, s.chunk_bytes);
  const bool chunks_apart = s.chunks == 1 || s.dst_chunk_stride >= s.chunk_bytes;
  const bool rows_apart = rows == 1 || s.dst_row_stride >= s.chunk_bytes;
  const bool by_row = chunks_apart && (rows == 1 || s.dst_row_stride >= row_span);
  const bool by_col = rows_apart && (s.chunks == 1 || s.dst_chunk_stride >= col_span);
  if (!by_row && !by_col) return MOE_E_ARG;
  if (s.src == s.dst) {
    if (rows > 1 && s.src_row_stride != s.dst_row_stride) return MOE_E_ARG;
    if (s.chunks > 1 && s.src_chunk_stride != s.dst_chunk_stride) return MOE_E_ARG;
    return MOE_OK;
  }
  const uintptr_t a = reinterpret_cast<uintptr_t>(s.src), b = reinterpret_cast<uintptr_t>(s.dst);
  if (a < b + (uintptr_t)dspan && b < a + (uintptr_t)sspan) return MOE_E_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_linear_q(const moe_linear* lin, const void* x, int64_t x_stride, int32_t T, void* y, int64_t y_stride,
                        void* stream) {
  MOE_TRY(check_linear(lin));
  if (T < 0) return MOE_E_ARG;
  if (T > kMaxTokens) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !y || !aligned(x, 16) || !aligned(y, act_size(lin->out))) return MOE_E_ARG;
  if (T > 1) {
    if (x_stride < lin->cols || y_stride < lin->rows || x_stride > kMaxStride || y_stride > kMaxStride)
      return MOE_E_ARG;
    if ((x_stride * (int64_t)act_size(lin->act)) % 16) return MOE_E_ARG;
  }
  const LinearArgs a{lin->w.codes, lin->w.scales, lin->w.mins, lin->bias, x, y, T > 1 ? x_stride : 0,
                     T > 1 ? y_stride : 0, T, lin->rows, lin->cols, lin->qfmt, lin->act, lin->out};
  return dev(launch_linear(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t moe_beam_workspace_bytes(const moe_beam* beam) {
  if (check_beam(beam) != MOE_OK) return 0;
  const size_t n = beam_ws_bytes(beam->batch, beam->beams, beam->vocab, beam->n_out, beam->act);
  return n ? n : 256;
}

moe_status moe_beam_select(const moe_beam* beam, const void* logits, int64_t logits_stride, const float* scores,
                           const uint8_t* finished_opt, const uint32_t* allowed_opt, int64_t allowed_stride,
                           float* out_score, int32_t* out_parent, int32_t* out_token, void* ws, size_t ws_bytes,
                           void* stream) {
  MOE_TRY(check_beam(beam));
  if (beam->batch == 0) return MOE_OK;
  if (!logits || !scores || !out_score || !out_parent || !out_token) return MOE_E_ARG;
  if (!aligned(logits, act_size(beam->act)) || !aligned(scores, 4) || !aligned(out_score, 4) ||
      !aligned(out_parent, 4) || !aligned(out_token, 4))
    return MOE_E_ARG;
  const int64_t rows = (int64_t)beam->batch * beam->beams;
  if (rows > 1 && (logits_stride < beam->vocab || logits_stride > kMaxStride)) return MOE_E_ARG;
  if (finished_opt && beam->eos < 0) return MOE_E_ARG;
  if (allowed_opt) {
    if (!aligned(allowed_opt, 4)) return MOE_E_ARG;
    if (allowed_stride != 0 && (allowed_stride < (beam->vocab + 31) / 32 || allowed_stride > kMaxStride))
      return MOE_E_ARG;
  }
  if (!ws) return MOE_E_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_E_ARG;
  if (ws_bytes < moe_beam_workspace_bytes(beam)) return MOE_E_WORKSPACE;
  const BeamArgs a{logits, rows > 1 ? logits_stride : 0, scores, finished_opt, allowed_opt, allowed_stride, out_score,
                   out_parent, out_token, ws, beam->batch, beam->beams, beam->vocab, beam->n_out, beam->act, beam->eos};
  return dev(launch_beam_select(a, reinterpret_cast<hipStream_t>(stream)));
}

moe_status moe_beam_reorder(const moe_state* states, int32_t n_states, const int32_t* parent, int64_t parent_stride,
                            int32_t batch, int32_t beams, void* stream) {
  if (n_states < 0 || batch < 0 || beams < 1) return MOE_E_ARG;
  if (beams > kMaxBeams || (int64_t)batch * beams > kMaxBeamRows) return MOE_E_UNSUPPORTED;
  if (n_states == 0 || batch == 0) return MOE_OK;
  if (!states || !parent || !aligned(parent, 4)) return MOE_E_ARG;
  if (batch > 1 && (parent_stride < beams || parent_stride > kMaxStride)) return MOE_E_ARG;
  for (int32_t i = 0; i < n_states; ++i) MOE_TRY(check_state(states[i], (int64_t)batch * beams));
  return dev(launch_beam_reorder(states, n_states, parent, batch > 1 ? parent_stride : 0, batch, beams,
                                 reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
