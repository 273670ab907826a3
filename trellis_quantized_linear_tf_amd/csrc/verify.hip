// Verification of drafted tokens against the target's logits, from given random numbers.
//
// A row's token is the first place whose running sum of weights w = exp((x - max) / T) is
// over u times their sum. Which place that is depends on sums over the whole row to the
// last bits, so weights and sums are in 64 bits. Rows are cut into chunks of kChunk
// logits, a wave each. The first launch reads every row once and leaves each chunk's
// maximum and sum (relative to its own maximum). The second finds, from a row's chunks,
// the one that the running sum crosses in, and reads only that one again.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

constexpr int kLane = 32;           // logits of a chunk a lane
constexpr int kChunk = 64 * kLane;  // 63.1 chunks of the head's 129280 columns: a lane each
constexpr int kWaves = 4;           // waves of a workgroup of independent waves
constexpr int kTreeWaves = 8;       // waves that share a sequence's rows
constexpr int kMaxNodes = 1024;

struct ChunkStat {
  double sum;  // of exp((x - top) / T); not set at T <= 0
  float top;   // largest logit, -inf if there is none
  int pad;
};

// What the chain's second launch leaves for the third, a sequence each.
struct ChainEnd {
  double z;
  float top;
  int row, first;
};

// 2^y for y <= 0 in 64 bits: 2^n 2^f with f = y - n in [-1/2, 1/2] and 2^f by the polynomial of
// degree 10 that equals it at the eleven Chebyshev nodes of that range (3.1e-16 relative).
__device__ __forceinline__ double pow2_poly(double f) {
  double p = 0x1.e6063f7217bc6p-28;
  p = __builtin_fma(p, f, 0x1.b675bca4eeebbp-24);
  p = __builtin_fma(p, f, 0x1.62bfd47773353p-20);
  p = __builtin_fma(p, f, 0x1.ffcb54062e698p-17);
  p = __builtin_fma(p, f, 0x1.430913096fd9fp-13);
  p = __builtin_fma(p, f, 0x1.5d87fe9d7a584p-10);
  p = __builtin_fma(p, f, 0x1.3b2ab6fba1ddap-7);
  p = __builtin_fma(p, f, 0x1.c6b08d703ce49p-5);
  p = __builtin_fma(p, f, 0x1.ebfbdff82c598p-3);
  p = __builtin_fma(p, f, 0x1.62e42fefa3a19p-1);
  return __builtin_fma(p, f, 1.0);
}

// For sums: what is below 2^-1000 (-inf and NaN too) counts as that, which no sum with a 1
// in it can tell from 0. Adding 1.5 2^52 rounds y to the integer n in the low word.
__device__ __forceinline__ double pow2_sum(double y) {
  y = fmax(y, -1000.0);
  const double t = y + 0x1.8p52;
  const double p = pow2_poly(y - (t - 0x1.8p52));
  const uint64_t bits = __builtin_bit_cast(uint64_t, p);
  const uint32_t hi = (uint32_t)(bits >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, t) << 20);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | (uint32_t)bits);
}

// The weight of logit x in a row of maximum top, s = log2(e) / T; 0 where it underflows.
__device__ __forceinline__ double weight_of(float x, float top, double s) {
  if (x == top) return 1.0;
  if (!(x > -INFINITY) || top == INFINITY) return 0.0;
  const double y = ((double)x - (double)top) * s;
  if (y < -1080.0) return 0.0;
  const double n = __builtin_rint(y);
  return __builtin_ldexp(pow2_poly(y - n), (int)n);
}

__device__ __forceinline__ double log2_scale(float temperature) { return 1.4426950408889634 / (double)temperature; }
__device__ __forceinline__ double fraction(float u) { return u > 0.f ? (double)u : 0.0; }

// A chunk's logits, -inf for NaN and behind the row's end. RUNS: a lane has kLane
// neighbours (for running sums); otherwise the lanes' pieces alternate.
template <int DT, bool RUNS>
__device__ __forceinline__ void load_chunk(const typename Elem<DT>::type* row, int64_t at, int vocab, float (&x)[kLane]) {
  constexpr int P = Elem<DT>::kPiece;
  const int lane = threadIdx.x & 63;
  if (at + kChunk <= vocab) {
    u32x4 v[kLane / P];
#pragma unroll
    for (int i = 0; i < kLane / P; ++i) v[i] = load_piece(row + at + (RUNS ? lane * kLane + i * P : (i * 64 + lane) * P));
#pragma unroll
    for (int i = 0; i < kLane / P; ++i) {
      float e[P];
      Elem<DT>::unpack(v[i], e);
#pragma unroll
      for (int c = 0; c < P; ++c) x[i * P + c] = e[c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      const int64_t j = at + (RUNS ? lane * kLane + i : i * 64 + lane);
      x[i] = -INFINITY;
      if (j < vocab) x[i] = Elem<DT>::load(row[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < kLane; ++i) x[i] = x[i] == x[i] ? x[i] : -INFINITY;
}

// Inclusive running sum over the wave's lanes.
__device__ __forceinline__ double wave_scan(double v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double up = __shfl_up(v, o);
    if (lane >= o) v += up;
  }
  return v;
}

template <int DT>
__device__ __forceinline__ const typename Elem<DT>::type* row_of(const VerifyArgs& a, int b, int i) {
  return static_cast<const typename Elem<DT>::type*>(a.logits) + b * a.stride_batch + i * a.stride_node;
}

// One wave per chunk of every row. Bound by the fp64 rate: some 22 full-rate operations
// a logit against 2 or 4 bytes.
template <int DT>
__global__ __launch_bounds__(kWaves * 64) void chunk_kernel(VerifyArgs a, int chunks) {
  const int64_t id = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6), row = id / chunks;
  if (row >= (int64_t)a.batch * a.nodes) return;
  const int b = (int)(row / a.nodes), chunk = (int)(id - row * chunks);
  float x[kLane];
  load_chunk<DT, false>(row_of<DT>(a, b, (int)(row - (int64_t)b * a.nodes)), (int64_t)chunk * kChunk, a.vocab, x);
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kLane; ++i) top = fmaxf(top, x[i]);
  top = wave_max(top);
  const float t = a.temperature ? a.temperature[b] : 1.f;
  double sum = 0.0;
  if (t > 0.f && top > -INFINITY) {
    double part[2] = {0.0, 0.0};
    if (top < INFINITY) {
      const double s = log2_scale(t), m = top;
#pragma unroll
      for (int i = 0; i < kLane; ++i) part[i & 1] += pow2_sum(((double)x[i] - m) * s);
    } else {
#pragma unroll
      for (int i = 0; i < kLane; ++i) part[i & 1] += x[i] == top ? 1.0 : 0.0;
    }
    sum = wave_sum(part[0] + part[1]);
  }
  if ((threadIdx.x & 63) == 0) static_cast<ChunkStat*>(a.workspace)[id] = {sum, top, 0};
}

__device__ __forceinline__ float row_top(const ChunkStat* stat, int chunks) {
  float top = -INFINITY;
  for (int c = threadIdx.x & 63; c < chunks; c += 64) top = fmaxf(top, stat[c].top);
  return wave_max(top);
}

__device__ __forceinline__ double row_sum(const ChunkStat* stat, int chunks, float top, double s) {
  double z = 0.0;
  for (int c = threadIdx.x & 63; c < chunks; c += 64) z += stat[c].sum * weight_of(stat[c].top, top, s);
  return wave_sum(z);
}

// First place of a row's maximum; top is above -inf.
template <int DT>
__device__ int first_place(const typename Elem<DT>::type* row, const ChunkStat* stat, int chunks, int vocab, float top) {
  const int lane = threadIdx.x & 63;
  int chunk = 0;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    const uint64_t hit = __ballot(c0 + lane < chunks && stat[c0 + lane < chunks ? c0 + lane : 0].top == top);
    if (hit) {
      chunk = c0 + __builtin_ctzll(hit);
      break;
    }
  }
  float x[kLane];
  load_chunk<DT, true>(row, (int64_t)chunk * kChunk, vocab, x);
  int mine = kLane;
#pragma unroll
  for (int i = kLane - 1; i >= 0; --i) mine = x[i] == top ? i : mine;
  const uint64_t hit = __ballot(mine < kLane);
  const int at = hit ? __builtin_ctzll(hit) : 0;
  return chunk * kChunk + at * kLane + __shfl(mine, at);
}

// Where the running sum of part(c), over the chunks c of a row, first is over goal: the
// chunk, and the sum before it. The last chunk of any weight where rounding lets none be.
template <typename F>
__device__ __forceinline__ int cross_chunk(int chunks, double goal, F part, double* before) {
  const int lane = threadIdx.x & 63;
  double base = 0.0, held = 0.0;
  int last = -1;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    const double v = c0 + lane < chunks ? part(c0 + lane) : 0.0;
    const double run = base + wave_scan(v);
    const uint64_t over = __ballot(v > 0.0 && run > goal), any = __ballot(v > 0.0);
    if (any) {
      const int at = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(any);
      const double up = __shfl(run, at > 0 ? at - 1 : 0);
      last = c0 + at;
      held = at > 0 ? up : base;
      if (over) break;
    }
    base = __shfl(run, 63);
  }
  *before = held;
  return last;
}

// The place in a chunk whose running sum, begun at before, first is over goal; the last
// place of any weight where rounding lets none be. w: the weights of the lane's run.
__device__ __forceinline__ int cross_place(const double (&w)[kLane], double before, double goal) {
  double mine = 0.0;
#pragma unroll
  for (int i = 0; i < kLane; ++i) mine += w[i];
  const double run = before + wave_scan(mine);
  const uint64_t over = __ballot(mine > 0.0 && run > goal), any = __ballot(mine > 0.0);
  const int at = over ? __builtin_ctzll(over) : any ? 63 - __builtin_clzll(any) : 0;
  double c = __shfl_up(run, 1);
  if ((threadIdx.x & 63) == 0) c = before;
  int place = -1, last = 0;
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    c += w[i];
    if (w[i] > 0.0) {
      last = i;
      if (place < 0 && c > goal) place = i;
    }
  }
  return at * kLane + __shfl(place < 0 ? last : place, at);
}

// A row's token, from its chunks; one wave, every lane gets it.
template <int DT>
__device__ int sample_row(const typename Elem<DT>::type* row, const ChunkStat* stat, int chunks, int vocab, float t, float u) {
  const float top = row_top(stat, chunks);
  if (top == -INFINITY) return -1;
  if (!(t > 0.f)) return first_place<DT>(row, stat, chunks, vocab, top);
  const double s = log2_scale(t);
  double before;
  const double goal = fraction(u) * row_sum(stat, chunks, top, s);
  const int chunk = cross_chunk(chunks, goal, [&](int c) { return stat[c].sum * weight_of(stat[c].top, top, s); }, &before);
  float x[kLane];
  load_chunk<DT, true>(row, (int64_t)chunk * kChunk, vocab, x);
  double w[kLane];
#pragma unroll
  for (int i = 0; i < kLane; ++i) w[i] = weight_of(x[i], top, s);
  return chunk * kChunk + cross_place(w, before, goal);
}

// One workgroup per sequence: its rows' tokens, a wave a row, then the first wave's walk.
template <int DT>
__global__ __launch_bounds__(kTreeWaves * 64) void tree_kernel(VerifyArgs a, int chunks) {
  __shared__ int token[kMaxNodes];
  const int b = blockIdx.x, lane = threadIdx.x & 63;
  const int64_t at = (int64_t)b * a.nodes;
  const float t = a.temperature ? a.temperature[b] : 1.f;
  const ChunkStat* stat = static_cast<const ChunkStat*>(a.workspace) + at * chunks;
  for (int i = threadIdx.x >> 6; i < a.nodes; i += kTreeWaves) {
    const int got = sample_row<DT>(row_of<DT>(a, b, i), stat + (int64_t)i * chunks, chunks, a.vocab, t, a.u[at + i]);
    if (lane == 0) token[i] = got;
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  int node = 0, count = 0;
  while (node >= 0) {
    if (lane == 0) a.accepted[at + count] = node;
    ++count;
    const int want = token[node];
    int next = -1;
    for (int c0 = node / 64 * 64; c0 < a.nodes && next < 0; c0 += 64) {
      const int c = c0 + lane;
      const uint64_t hit = __ballot(c > node && c < a.nodes && want >= 0 && a.parents[at + (c < a.nodes ? c : 0)] == node &&
                                    a.tokens[at + (c < a.nodes ? c : 0)] == want);
      if (hit) next = c0 + __builtin_ctzll(hit);
    }
    if (next < 0 && lane == 0) {
      a.count[b] = count;
      a.next[b] = want;
    }
    node = next;
  }
  for (int c = count + lane; c < a.nodes; c += 64) a.accepted[at + c] = -1;
}

struct Row {
  float top;
  int first;  // of the maximum, at T <= 0
  double z;
};

template <int DT>
__device__ __forceinline__ Row row_stat(const VerifyArgs& a, int chunks, int b, int j, float t) {
  const ChunkStat* stat = static_cast<const ChunkStat*>(a.workspace) + ((int64_t)b * a.nodes + j) * chunks;
  Row r = {row_top(stat, chunks), -1, 0.0};
  if (r.top == -INFINITY) return r;
  if (t > 0.f) {
    r.z = row_sum(stat, chunks, r.top, log2_scale(t));
  } else {
    r.first = first_place<DT>(row_of<DT>(a, b, j), stat, chunks, a.vocab, r.top);
    r.z = 1.0;
  }
  return r;
}

// Probability of place i with logit x; s is not used at T <= 0.
__device__ __forceinline__ double probability(const Row& r, float t, double s, int i, float x) {
  if (!(t > 0.f)) return i == r.first ? 1.0 : 0.0;
  return r.z > 0.0 ? weight_of(x == x ? x : -INFINITY, r.top, s) / r.z : 0.0;
}

// max(p - q, 0) of the lane's part of a chunk (p where q is NULL).
template <int DT, bool RUNS>
__device__ __forceinline__ void residual(const typename Elem<DT>::type* row, const float* q, const Row& r, float t, int64_t at,
                                         int vocab, double (&w)[kLane]) {
  constexpr int P = Elem<DT>::kPiece;
  const int lane = threadIdx.x & 63;
  const double s = t > 0.f ? log2_scale(t) : 0.0;
  const bool whole = at + kChunk <= vocab;  // as load_chunk goes
  float x[kLane];
  load_chunk<DT, RUNS>(row, at, vocab, x);
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    const int64_t j = at + (RUNS ? lane * kLane + i : whole ? (i / P * 64 + lane) * P + i % P : i * 64 + lane);
    double p = probability(r, t, s, (int)j, x[i]);
    if (q != nullptr && j < vocab) p -= (double)q[j];
    w[i] = p > 0.0 && j < vocab ? p : 0.0;
  }
}

// One workgroup per sequence and group of chunks: goes down the drafts to the first that
// is refused, then sums max(p - q, 0) over its chunks of that row, a wave each. Every
// workgroup of a sequence takes the same way.
template <int DT>
__global__ __launch_bounds__(kWaves * 64) void chain_kernel(VerifyArgs a, int chunks, double* sums, ChainEnd* ends) {
  __shared__ int refused[kWaves];
  __shared__ Row rows[kWaves];
  const int b = blockIdx.y, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t at = (int64_t)b * a.nodes;
  const float t = a.temperature ? a.temperature[b] : 1.f;
  int stop = -1;
  for (int j0 = 0; stop < 0; j0 += kWaves) {
    const int j = j0 + wave;
    int no = 0;
    Row r = {-INFINITY, -1, 0.0};
    if (j < a.nodes) {
      r = row_stat<DT>(a, chunks, b, j, t);
      no = 1;  // the last row has no draft
      if (j + 1 < a.nodes) {
        const int x = a.tokens[at + j + 1];
        if (x >= 0 && x < a.vocab) {
          const double p = probability(r, t, t > 0.f ? log2_scale(t) : 0.0, x, Elem<DT>::load(row_of<DT>(a, b, j)[x]));
          const float q = a.q[b * a.q_stride_batch + j * a.q_stride_node + x];
          no = !(fraction(a.u[at + j]) * (double)q < p);
        }
      }
    }
    __syncthreads();
    if (lane == 0) {
      refused[wave] = no;
      rows[wave] = r;
    }
    __syncthreads();
    for (int w = kWaves - 1; w >= 0; --w)
      if (refused[w]) stop = j0 + w;
  }
  const Row r = rows[stop % kWaves];
  const int chunk = blockIdx.x * kWaves + wave;
  if (blockIdx.x == 0 && threadIdx.x == 0) ends[b] = {r.z, r.top, stop, r.first};
  if (chunk >= chunks || stop + 1 == a.nodes) return;
  double w[kLane], sum = 0.0;
  residual<DT, false>(row_of<DT>(a, b, stop), a.q + b * a.q_stride_batch + stop * a.q_stride_node, r, t,
                      (int64_t)chunk * kChunk, a.vocab, w);
#pragma unroll
  for (int i = 0; i < kLane; ++i) sum += w[i];
  sum = wave_sum(sum);
  if (lane == 0) sums[(int64_t)b * chunks + chunk] = sum;
}

// One wave per sequence: the token after the accepted drafts.
template <int DT>
__global__ __launch_bounds__(64) void chain_next_kernel(VerifyArgs a, int chunks, const double* sums, const ChainEnd* ends) {
  const int b = blockIdx.x, lane = threadIdx.x;
  const ChainEnd end = ends[b];
  const float t = a.temperature ? a.temperature[b] : 1.f, u = a.u[(int64_t)b * a.nodes + a.nodes - 1];
  const auto* row = row_of<DT>(a, b, end.row);
  double total = 0.0;
  if (end.row + 1 < a.nodes)
    for (int c = lane; c < chunks; c += 64) total += sums[(int64_t)b * chunks + c];
  total = wave_sum(total);
  int place;
  if (total > 0.0) {
    double before, w[kLane];
    const double goal = fraction(u) * total;
    const int chunk = cross_chunk(chunks, goal, [&](int c) { return sums[(int64_t)b * chunks + c]; }, &before);
    residual<DT, true>(row, a.q + b * a.q_stride_batch + end.row * a.q_stride_node, {end.top, end.first, end.z}, t,
                       (int64_t)chunk * kChunk, a.vocab, w);
    place = chunk * kChunk + cross_place(w, before, goal);
  } else {
    const ChunkStat* stat = static_cast<const ChunkStat*>(a.workspace) + ((int64_t)b * a.nodes + end.row) * chunks;
    place = sample_row<DT>(row, stat, chunks, a.vocab, t, u);
  }
  if (lane == 0) {
    a.count[b] = end.row + 1;
    a.next[b] = place;
  }
}

static int chunks_of(int vocab) { return (int)(((int64_t)vocab + kChunk - 1) / kChunk); }

template <int DT>
static hipError_t launch(const VerifyArgs& a, hipStream_t stream) {
  const int chunks = chunks_of(a.vocab);
  const int64_t rows = (int64_t)a.batch * a.nodes, groups = (rows * chunks + kWaves - 1) / kWaves;
  if (groups > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(chunk_kernel<DT>, dim3((unsigned)groups), dim3(kWaves * 64), 0, stream, a, chunks);
  if (a.parents != nullptr) {
    hipLaunchKernelGGL(tree_kernel<DT>, dim3(a.batch), dim3(kTreeWaves * 64), 0, stream, a, chunks);
  } else {
    double* sums = reinterpret_cast<double*>(static_cast<ChunkStat*>(a.workspace) + rows * chunks);
    ChainEnd* ends = reinterpret_cast<ChainEnd*>(sums + (int64_t)a.batch * chunks);
    hipLaunchKernelGGL(chain_kernel<DT>, dim3((chunks + kWaves - 1) / kWaves, a.batch), dim3(kWaves * 64), 0, stream, a, chunks,
                       sums, ends);
    hipLaunchKernelGGL(chain_next_kernel<DT>, dim3(a.batch), dim3(64), 0, stream, a, chunks, sums, ends);
  }
  return hipGetLastError();
}

size_t verify_workspace(int batch, int nodes, int vocab) {
  const size_t chunks = (size_t)chunks_of(vocab), b = (size_t)(batch < 1 ? 1 : batch);
  return (b * nodes * chunks * sizeof(ChunkStat) + b * chunks * sizeof(double) + b * sizeof(ChainEnd) + 15) / 16 * 16;
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
  if (a.dtype == TF_DT_F32) return launch<TF_DT_F32>(a, stream);
  if (a.dtype == TF_DT_F16) return launch<TF_DT_F16>(a, stream);
  return launch<TF_DT_BF16>(a, stream);
}

}  // namespace tf_exl3
