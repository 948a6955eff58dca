// Beam search: the n best continuations of each sequence over beams and
// vocabulary, and the move of the beams' states to follow their parents.
//
// Selection.  k_beam_rows: one block per beam evaluates L = log sum exp over
// the allowed logits (maximum, then the sum of exp(l - max) in 64 bits) and
// picks the row's n largest logits one after the other (equal logits: lower
// token).  k_beam_merge: one block per sequence picks the n largest of the
// beams' candidates by total = score + (logit - L) in 64 bits.
#include "moe_device.h"
#include "moe_internal.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct RowList {   // workspace of one selection
  double* lse;     // [B*W], NaN: the row has no candidates
  uint64_t* keys;  // [B*W][n] sel_key(logit, token), 0 past the last
};

__host__ __device__ inline RowList row_list(void* ws, int rows) {
  const size_t at = ((size_t)rows * 8 + 255) & ~(size_t)255;
  return RowList{reinterpret_cast<double*>(ws), reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(ws) + at)};
}

__device__ __forceinline__ bool allowed(const BeamArgs& a, int row, int v) {
  return !a.allowed || ((a.allowed[(size_t)row * a.ld_allowed + (v >> 5)] >> (v & 31)) & 1u);
}

// (+ 0: a negative zero equals a positive one and must not sort below it)
template <int ACT>
__device__ __forceinline__ float logit(const BeamArgs& a, int row, int v) {
  return allowed(a, row, v) ? load_act<ACT>(a.logits, (size_t)row * a.ld + v) + 0.0f : -INFINITY;
}

// Block-wide maximum of a 64-bit key / sum of a double (every thread gets it).
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* sh) {
  v = wave_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int i = 0; i < kThreads / 64; ++i) v = sh[i] > v ? sh[i] : v;
  return v;
}
__device__ __forceinline__ double block_sum(double v, double* sh) {
  __syncthreads();
  sh[threadIdx.x] = v;
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if ((int)threadIdx.x < s) sh[threadIdx.x] += sh[threadIdx.x + s];
    __syncthreads();
  }
  return sh[0];
}

template <int ACT>
__global__ __launch_bounds__(kThreads) void k_beam_rows(BeamArgs a) {
  __shared__ double dsh[kThreads];
  __shared__ uint64_t ksh[kThreads / 64];
  const int row = blockIdx.x;
  if (a.finished && a.finished[row]) return;  // its one candidate needs no logits
  const RowList out = row_list(a.ws, a.B * a.W);
  uint64_t best = 0;
  bool bad = false;
  for (int v = threadIdx.x; v < a.V; v += kThreads) {
    const float l = logit<ACT>(a, row, v);
    if (l != l || l == INFINITY) bad = true;
    const uint64_t k = sel_key(l, v);
    best = k > best ? k : best;
  }
  const bool any_bad = __syncthreads_or(bad);
  best = block_max(best, ksh);
  const float top = key_value((uint32_t)(best >> 32));
  const bool none = any_bad || top == -INFINITY;
  double sum = 0.0;
  if (!none)
    for (int v = threadIdx.x; v < a.V; v += kThreads) sum += exp((double)logit<ACT>(a, row, v) - (double)top);
  sum = block_sum(sum, dsh);
  if (threadIdx.x == 0) out.lse[row] = none ? __longlong_as_double(0x7ff8000000000000ll) : (double)top + log(sum);
  if (none) return;
  for (int i = 0; i < a.n; ++i) {
    if (threadIdx.x == 0) out.keys[(size_t)row * a.n + i] = best;
    if (best == 0) continue;
    const uint64_t last = best;
    best = 0;
    for (int v = threadIdx.x; v < a.V; v += kThreads) {
      const float l = logit<ACT>(a, row, v);
      const uint64_t k = l == -INFINITY ? 0 : sel_key(l, v);
      if (k < last && k > best) best = k;
    }
    best = block_max(best, ksh);
  }
}

// Order-preserving map of a double (never NaN here).
__device__ __forceinline__ uint64_t order_key64(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key64_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// Candidate i of beam w: its total (as an ordered key, 0: none) and token.
__device__ __forceinline__ uint64_t candidate(const BeamArgs& a, const RowList& in, int row, int i, int* token) {
  const float s = a.scores[row];
  if (!(s > -INFINITY && s < INFINITY)) return 0;
  if (a.finished && a.finished[row]) {
    *token = a.eos;
    return i == 0 ? order_key64((double)s) : 0;
  }
  const double L = in.lse[row];
  if (L != L) return 0;
  const uint64_t k = in.keys[(size_t)row * a.n + i];
  if (k == 0) return 0;
  *token = key_id(k);
  return order_key64((double)s + ((double)key_value((uint32_t)(k >> 32)) - L));
}

__global__ __launch_bounds__(kThreads) void k_beam_merge(BeamArgs a) {
  __shared__ uint64_t ksh[kThreads / 64];
  const int b = blockIdx.x;
  const RowList in = row_list(a.ws, a.B * a.W);
  const int total = a.W * a.n;
  uint64_t last = ~0ull;
  uint32_t last_flat = 0;
  for (int o = 0; o < a.n; ++o) {
    // the largest key below (last, last_flat) in the order (key desc, flat asc)
    uint64_t best = 0;
    for (int c = threadIdx.x; c < total; c += kThreads) {
      int token = 0;
      const int w = c / a.n;
      const uint64_t k = candidate(a, in, b * a.W + w, c % a.n, &token);
      const uint32_t flat = (uint32_t)w * (uint32_t)a.V + (uint32_t)token;
      if (k && (k < last || (k == last && flat > last_flat)) && k > best) best = k;
    }
    best = block_max(best, ksh);
    uint64_t low = 0;  // lowest flat index at that key, as ~flat + 1
    if (best)
      for (int c = threadIdx.x; c < total; c += kThreads) {
        int token = 0;
        const int w = c / a.n;
        const uint64_t k = candidate(a, in, b * a.W + w, c % a.n, &token);
        const uint32_t flat = (uint32_t)w * (uint32_t)a.V + (uint32_t)token;
        if (k == best && (k < last || flat > last_flat)) {
          const uint64_t inv = (uint64_t)(0xffffffffu - flat) + 1;
          low = inv > low ? inv : low;
        }
      }
    low = block_max(low, ksh);
    const size_t at = (size_t)b * a.n + o;
    const uint32_t flat = 0xffffffffu - (uint32_t)(low - 1);
    if (threadIdx.x == 0) {
      a.out_score[at] = best ? (float)key64_value(best) : -INFINITY;
      a.out_parent[at] = best ? (int)(flat / (uint32_t)a.V) : -1;
      a.out_token[at] = best ? (int)(flat % (uint32_t)a.V) : -1;
    }
    last = best;
    last_flat = flat;
    if (!best) last = 0;
  }
}

// ---------------------------------------------------------------- reordering
constexpr int kStates = 32;  // states per launch (the descriptors travel as kernel arguments)

struct StateArgs {
  moe_state s[kStates];
  const int32_t* parent;
  int64_t ldp;
  int W;
};

// Block (x, sequence, state): each thread owns columns (byte positions) of
// every row of one sequence, reads the column of all parents before it writes
// any, and nobody else touches that column, so dst may be src.
__global__ __launch_bounds__(kThreads) void k_reorder(StateArgs a) {
  const moe_state& s = a.s[blockIdx.z];
  const int b = blockIdx.y;
  const int64_t total = s.chunks * s.chunk_bytes;
  const char* src = reinterpret_cast<const char*>(s.src) + (int64_t)b * a.W * s.src_row_stride;
  char* dst = reinterpret_cast<char*>(s.dst) + (int64_t)b * a.W * s.dst_row_stride;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < total; c += (int64_t)gridDim.x * kThreads) {
    const int64_t piece = c / s.chunk_bytes, off = c % s.chunk_bytes;
    char v[64];
    for (int i = 0; i < a.W; ++i) {
      const int p = a.parent[b * a.ldp + i];
      v[i] = p >= 0 && p < a.W ? src[p * s.src_row_stride + piece * s.src_chunk_stride + off] : 0;
    }
    for (int i = 0; i < a.W; ++i) {
      const int p = a.parent[b * a.ldp + i];
      if (p >= 0 && p < a.W) dst[i * s.dst_row_stride + piece * s.dst_chunk_stride + off] = v[i];
    }
  }
}

}  // namespace

size_t beam_ws_bytes(int B, int W, int V, int n, int act) {
  (void)V; (void)act;
  const size_t rows = (size_t)B * W;
  return ((rows * 8 + 255) & ~(size_t)255) + ((rows * n * 8 + 255) & ~(size_t)255);
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
  const unsigned rows = (unsigned)(a.B * a.W);
  if (a.act == MOE_ACT_BF16) k_beam_rows<MOE_ACT_BF16><<<rows, kThreads, 0, s>>>(a);
  else k_beam_rows<MOE_ACT_F32><<<rows, kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_beam_merge<<<(unsigned)a.B, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const moe_state* states, int n, const int32_t* parent, int64_t ldp, int B, int W,
                               hipStream_t s) {
  for (int b0 = 0; b0 < B; b0 += 65535) {
    const int nb = B - b0 < 65535 ? B - b0 : 65535;
    StateArgs a{};
    a.parent = parent + b0 * ldp;
    a.ldp = ldp;
    a.W = W;
    int m = 0;
    int64_t most = 0;
    for (int i = 0; i < n; ++i) {
      moe_state st = states[i];
      if (st.chunk_bytes && st.chunks) {
        if (B * W == 1) st.src_row_stride = st.dst_row_stride = 0;
        if (st.chunks == 1) st.src_chunk_stride = st.dst_chunk_stride = 0;
        st.src = reinterpret_cast<const char*>(st.src) + (int64_t)b0 * W * st.src_row_stride;
        st.dst = reinterpret_cast<char*>(st.dst) + (int64_t)b0 * W * st.dst_row_stride;
        most = st.chunks * st.chunk_bytes > most ? st.chunks * st.chunk_bytes : most;
        a.s[m++] = st;
      }
      if (m == kStates || (i == n - 1 && m > 0)) {
        const int64_t want = (most + kThreads - 1) / kThreads;
        const dim3 grid((unsigned)(want < 1024 ? want : 1024), (unsigned)nb, (unsigned)m);
        k_reorder<<<grid, kThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        m = 0;
        most = 0;
      }
    }
  }
  return hipSuccess;
}

}  // namespace moe
