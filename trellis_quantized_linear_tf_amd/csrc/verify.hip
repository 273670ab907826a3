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
constexpr int kSampleThreads = 256;  // of the workgroup that looks through one chunk
constexpr int kRun = kChunk / kSampleThreads;
constexpr int kChainWaves = 8;

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

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 2^y for y <= 0 in 64 bits: 2^n 2^f with f = y - n in [-1/2, 1/2] and 2^f = 1 + f g(f), g the
// polynomial of degree 9 that equals (2^f - 1) / f at the ten Chebyshev nodes of that range: 5.7e-16
// relative at most, to both sides alike, and exact at 0.
__device__ __forceinline__ double pow2_poly(double f) {
  double p = 0x1.e5e9f548e5725p-28;
  p = __builtin_fma(p, f, 0x1.b6571de2f2351p-24);
  p = __builtin_fma(p, f, 0x1.62bfe46117445p-20);
  p = __builtin_fma(p, f, 0x1.ffcb76789860fp-17);
  p = __builtin_fma(p, f, 0x1.4309130378460p-13);
  p = __builtin_fma(p, f, 0x1.5d87fe908f88ap-10);
  p = __builtin_fma(p, f, 0x1.3b2ab6fba385fp-7);
  p = __builtin_fma(p, f, 0x1.c6b08d7044119p-5);
  p = __builtin_fma(p, f, 0x1.ebfbdff82c590p-3);
  p = __builtin_fma(p, f, 0x1.62e42fefa39f7p-1);
  return __builtin_fma(p, f, 1.0);
}

// For sums, 64 table entries 2^(j / 64), j = 0 .. 63, in shared memory shorten that: with y = (64 n + j
// + r) / 64, 2^y = 2^n 2^(j / 64) 2^(r / 64), the last by a polynomial of degree 4 (2.4e-15 relative at
// most, to both sides alike). A running sum is off by less than 3e-15 of the row's sum and the sums' own
// roundings, which over a row of 129280 moves it past a random number with a chance of 1e-9 at most.
// What is below 2^-1000 (-inf and NaN too) counts as that, which no sum with a 1 in it can tell
// from 0. Adding 1.5 2^52 rounds 64 y to an integer in the low word; shifted by 14 bits it adds n to the
// exponent, and j 2^14 which the entries have been lowered by.
constexpr int kTable = 64;

__device__ __forceinline__ void fill_table(double* table) {
  if (threadIdx.x < kTable) {
    u32x2 w = __builtin_bit_cast(u32x2, exp2((double)threadIdx.x / kTable));
    w[1] -= threadIdx.x << 14;
    table[threadIdx.x] = __builtin_bit_cast(double, w);
  }
  __syncthreads();
}

// sum + 2^y by y64 = 64 y.
__device__ __forceinline__ double add_pow2(double sum, double y64, const double* table) {
  y64 = fmax(y64, -64000.0);
  const double t = y64 + 0x1.8p52, r = y64 - (t - 0x1.8p52);
  const uint32_t n = __builtin_bit_cast(u32x2, t)[0];
  u32x2 w = __builtin_bit_cast(u32x2, table[n % kTable]);
  w[1] += n << 14;
  double p = 0x1.3b2ad0385b409p-31;
  p = __builtin_fma(p, r, 0x1.c6b0c40d8c4e9p-23);
  p = __builtin_fma(p, r, 0x1.ebfbdff82ac52p-15);
  p = __builtin_fma(p, r, 0x1.62e42fefa0352p-7);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_fma(__builtin_bit_cast(double, w), p, sum);
}

// The same for one: what is below 2^-1000 counts as 0.
__device__ __forceinline__ double pow2_or_0(double y) {
  if (!(y > -1000.0)) return 0.0;
  const double t = y + 0x1.8p52;
  u32x2 w = __builtin_bit_cast(u32x2, pow2_poly(y - (t - 0x1.8p52)));
  w[1] += __builtin_bit_cast(u32x2, t)[0] << 20;
  return __builtin_bit_cast(double, w);
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

// A wave's chunk, -inf behind the row's end; the lanes' pieces of 16 bytes alternate. Element
// i of a lane stands at `place`.
template <int DT>
__device__ __forceinline__ int64_t place(int64_t at, int vocab, int i) {
  constexpr int P = Elem<DT>::kPiece;
  const int lane = threadIdx.x & 63;
  return at + (at + kChunk <= vocab ? (i / P * 64 + lane) * P + i % P : i * 64 + lane);
}

template <int DT>
__device__ __forceinline__ void load_chunk(const typename Elem<DT>::type* row, int64_t at, int vocab, float (&x)[kLane]) {
  constexpr int P = Elem<DT>::kPiece;
  const int lane = threadIdx.x & 63;
  if (at + kChunk <= vocab) {
    u32x4 v[kLane / P];
#pragma unroll
    for (int i = 0; i < kLane / P; ++i) v[i] = load_piece(row + at + (i * 64 + lane) * P);
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
      const int64_t j = at + i * 64 + lane;
      x[i] = -INFINITY;
      if (j < vocab) x[i] = Elem<DT>::load(row[j]);
    }
  }
}

// A thread's kRun neighbours of a workgroup's chunk, -inf behind the row's end.
template <int DT>
__device__ __forceinline__ void load_run(const typename Elem<DT>::type* row, int64_t at, int vocab, float (&x)[kRun]) {
  constexpr int P = Elem<DT>::kPiece;
  if (at + kRun <= vocab) {
#pragma unroll
    for (int i = 0; i < kRun / P; ++i) {
      float e[P];
      Elem<DT>::unpack(load_piece(row + at + i * P), e);
#pragma unroll
      for (int c = 0; c < P; ++c) x[i * P + c] = e[c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) x[i] = at + i < vocab ? Elem<DT>::load(row[at + i]) : -INFINITY;
  }
}

template <int DT>
__device__ __forceinline__ const typename Elem<DT>::type* row_of(const VerifyArgs& a, int b, int i) {
  return static_cast<const typename Elem<DT>::type*>(a.logits) + b * a.stride_batch + i * a.stride_node;
}

// One wave per chunk of every row. Bound by the fp64 rate: some 17 full-rate operations
// a logit against 2 or 4 bytes: 768 rows of 129280 bf16 58 us (by a polynomial of degree 9 and no
// table 62, with 98% of the cycles issuing vector instructions); 512 rows of fp32 44 us, 6.0 TB/s.
// Workgroups of 8 or 16 waves, or several chunks a wave, share the table more and measured
// 58 to 63 us.
template <int DT>
__global__ __launch_bounds__(kWaves * 64) void chunk_kernel(VerifyArgs a, int chunks) {
  __shared__ double table[kTable];
  const int64_t id = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6), row = id / chunks;
  const bool there = row < (int64_t)a.batch * a.nodes;
  const int b = (int)(row / a.nodes), chunk = (int)(id - row * chunks);
  float x[kLane];
  // fp32 rows are bound by their bytes and are on their way before the table is made (43 us against
  // 45 in the case above); 16-bit rows by their instructions, and kept longer they cost more (61 against 57).
  if (DT != TF_DT_F32) fill_table(table);
  if (there) load_chunk<DT>(row_of<DT>(a, b, (int)(row - (int64_t)b * a.nodes)), (int64_t)chunk * kChunk, a.vocab, x);
  if (DT == TF_DT_F32) fill_table(table);
  if (!there) return;
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kLane; ++i) top = fmaxf(top, x[i]);
  top = wave_max(top);
  const float t = a.temperature ? a.temperature[b] : 1.f;
  double sum = 0.0;
  if (t > 0.f && top > -INFINITY) {
    if (top < INFINITY) {
      const double s = log2_scale(t) * kTable, m = top;
#pragma unroll
      for (int i = 0; i < kLane; ++i) sum = add_pow2(sum, ((double)x[i] - m) * s, table);
    } else {
#pragma unroll
      for (int i = 0; i < kLane; ++i) sum += x[i] == top ? 1.0 : 0.0;
    }
    sum = wave_sum(sum);
  }
  if ((threadIdx.x & 63) == 0) static_cast<ChunkStat*>(a.workspace)[id] = {sum, top, 0};
}

// Where the running sum of part(c) over a row's chunks first is over u times its total; at
// the last chunk of any weight if rounding lets none be. One wave, or each of several.
struct Cross {
  int chunk;  // -1: no weight at all
  double before, goal;
};

template <typename F>
__device__ __forceinline__ Cross cross_chunk(int chunks, double u, F part) {
  const int lane = threadIdx.x & 63;
  double base = 0.0, v = 0.0, run = 0.0;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    v = c0 + lane < chunks ? part(c0 + lane) : 0.0;
    run = base + wave_scan(v);
    base = lane_of(run, 63);
  }
  Cross x = {-1, 0.0, u * base};
  base = 0.0;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    if (chunks > 64) {  // otherwise at hand
      v = c0 + lane < chunks ? part(c0 + lane) : 0.0;
      run = base + wave_scan(v);
    }
    const uint64_t over = __ballot(v > 0.0 && run > x.goal), any = __ballot(v > 0.0);
    if (any) {
      const int at = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(any);
      x.chunk = c0 + at;
      x.before = at > 0 ? lane_of(run, at - 1) : base;
      if (over) break;
    }
    base = lane_of(run, 63);
  }
  return x;
}

__device__ __forceinline__ float row_top(const ChunkStat* stat, int chunks) {
  float top = -INFINITY;
  for (int c = threadIdx.x & 63; c < chunks; c += 64) top = fmaxf(top, stat[c].top);
  return wave_max(top);
}

// First chunk of a row that holds its maximum.
__device__ __forceinline__ int top_chunk(const ChunkStat* stat, int chunks, float top) {
  const int lane = threadIdx.x & 63;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    const uint64_t hit = __ballot(c0 + lane < chunks && stat[c0 + lane < chunks ? c0 + lane : 0].top == top);
    if (hit) return c0 + __builtin_ctzll(hit);
  }
  return 0;
}

struct Found {
  double sum[kSampleThreads / 64];
  int first[kSampleThreads / 64], last[kSampleThreads / 64];
};

// The place in a workgroup's chunk, whose threads hold the weights w of their runs, where
// the running sum, begun at before, first is over goal; the last place of any weight if
// rounding lets none be.
__device__ __forceinline__ int cross_place(const double (&w)[kRun], double before, double goal, Found& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double mine = 0.0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) mine += w[i];
  const double scan = wave_scan(mine);
  if (lane == 63) f.sum[wave] = scan;
  __syncthreads();
  for (int i = 0; i < wave; ++i) before += f.sum[i];
  const double run = before + scan;
  double c = run - mine;
  int over = kRun, last = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    c += w[i];
    if (w[i] > 0.0) {
      last = i;
      if (over == kRun && c > goal) over = i;
    }
  }
  const uint64_t hit = __ballot(mine > 0.0 && run > goal), any = __ballot(mine > 0.0);
  if (lane == 0) f.first[wave] = f.last[wave] = -1;
  const int from = threadIdx.x * kRun;
  if (hit && lane == __builtin_ctzll(hit)) f.first[wave] = from + (over < kRun ? over : last);
  if (any && lane == 63 - __builtin_clzll(any)) f.last[wave] = from + last;
  __syncthreads();
  int at = 0;
  for (int i = 0; i < kSampleThreads / 64; ++i)
    if (f.last[i] >= 0) at = f.last[i];
  for (int i = kSampleThreads / 64 - 1; i >= 0; --i)
    if (f.first[i] >= 0) at = f.first[i];
  return at;
}

// A row's token from its chunks; one workgroup, every thread gets it.
template <int DT>
__device__ __forceinline__ int sample_row(const typename Elem<DT>::type* row, const ChunkStat* stat, int chunks, int vocab, float t,
                                          float u, Found& f) {
  const float top = row_top(stat, chunks);
  if (top == -INFINITY) return -1;
  float x[kRun];
  double w[kRun];
  Cross at = {0, 0.0, 0.0};
  if (t > 0.f) {
    const double s = log2_scale(t);
    at = cross_chunk(chunks, fraction(u), [&](int c) { return stat[c].sum * weight_of(stat[c].top, top, s); });
    load_run<DT>(row, (int64_t)at.chunk * kChunk + threadIdx.x * kRun, vocab, x);
#pragma unroll
    for (int i = 0; i < kRun; ++i) w[i] = weight_of(x[i], top, s);
  } else {
    at.chunk = top_chunk(stat, chunks, top);
    load_run<DT>(row, (int64_t)at.chunk * kChunk + threadIdx.x * kRun, vocab, x);
#pragma unroll
    for (int i = 0; i < kRun; ++i) w[i] = x[i] == top ? 1.0 : 0.0;
  }
  return at.chunk * kChunk + cross_place(w, at.before, at.goal, f);
}

// One workgroup per row: its token.
template <int DT>
__global__ __launch_bounds__(kSampleThreads) void token_kernel(VerifyArgs a, int chunks, int32_t* token) {
  __shared__ Found f;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / a.nodes), i = (int)(row - (int64_t)b * a.nodes);
  const int got = sample_row<DT>(row_of<DT>(a, b, i), static_cast<const ChunkStat*>(a.workspace) + row * chunks, chunks, a.vocab,
                                 a.temperature ? a.temperature[b] : 1.f, a.u[row], f);
  if (threadIdx.x == 0) token[row] = got;
}

// One wave per sequence walks its tree, 64 nodes looked at together.
__global__ __launch_bounds__(64) void walk_kernel(VerifyArgs a, const int32_t* token) {
  const int b = blockIdx.x, lane = threadIdx.x;
  const int64_t at = (int64_t)b * a.nodes;
  int parent = -1, mine = -1, row_token = -1;  // of node `lane`, for trees of up to 64
  if (lane < a.nodes) parent = a.parents[at + lane], mine = a.tokens[at + lane], row_token = token[at + lane];
  int node = 0, count = 0;
  while (node >= 0) {
    if (lane == 0) a.accepted[at + count] = node;
    ++count;
    const int want = node < 64 ? __builtin_amdgcn_readlane(row_token, node) : token[at + node];
    int next = -1;
    for (int c0 = node / 64 * 64; c0 < a.nodes && next < 0; c0 += 64) {
      const int c = c0 + lane, have = c < a.nodes ? c : 0;
      const bool child = c0 == 0 ? parent == node && mine == want : a.parents[at + have] == node && a.tokens[at + have] == want;
      const uint64_t hit = __ballot(c > node && c < a.nodes && want >= 0 && child);
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

// A row's maximum with its sum or, at T <= 0, its first place; one wave.
template <int DT>
__device__ __forceinline__ Row row_stat(const VerifyArgs& a, int chunks, int b, int j, float t) {
  const ChunkStat* stat = static_cast<const ChunkStat*>(a.workspace) + ((int64_t)b * a.nodes + j) * chunks;
  Row r = {row_top(stat, chunks), -1, 0.0};
  if (r.top == -INFINITY) return r;
  if (t > 0.f) {
    const double s = log2_scale(t);
    double z = 0.0;
    for (int c = threadIdx.x & 63; c < chunks; c += 64) z += stat[c].sum * weight_of(stat[c].top, r.top, s);
    r.z = wave_sum(z);
  } else {
    const int64_t at = (int64_t)top_chunk(stat, chunks, r.top) * kChunk;
    float x[kLane];
    load_chunk<DT>(row_of<DT>(a, b, j), at, a.vocab, x);
    int64_t first = 0x7FFFFFFF;
#pragma unroll
    for (int i = kLane - 1; i >= 0; --i) first = x[i] == r.top ? place<DT>(at, a.vocab, i) : first;
    int low = (int)first;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) low = min(low, __shfl_xor(low, o));
    r.first = low;
    r.z = 1.0;
  }
  return r;
}

// Probability of place i with logit x; s = log2(e) / T, not used at T <= 0.
__device__ __forceinline__ double probability(const Row& r, float t, double s, int i, float x) {
  if (!(t > 0.f)) return i == r.first ? 1.0 : 0.0;
  return r.z > 0.0 ? weight_of(x, r.top, s) / r.z : 0.0;
}

// The same by the reciprocal of the sum, for residuals: where p and q, which has 24 bits, can
// be equal at all (a power of two) the product is as exact as the quotient.
__device__ __forceinline__ double residual(const Row& r, double s, double inv, float x, float q) {
  const double d = weight_of(x, r.top, s) * inv - (double)q;
  return d > 0.0 ? d : 0.0;
}

// One workgroup per sequence and group of chunks: goes down the drafts to the first that
// is refused, a wave a row, then sums max(p - q, 0) over its chunks of that row, a wave each.
// Every workgroup of a sequence takes the same way. At T <= 0 there is nothing to sum: p
// is 1 at one place, which is the token whatever q holds.
template <int DT>
__global__ __launch_bounds__(kChainWaves * 64) void chain_kernel(VerifyArgs a, int chunks, double* sums, ChainEnd* ends) {
  __shared__ int refused[kChainWaves];
  __shared__ Row rows[kChainWaves];
  const int b = blockIdx.y, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t at = (int64_t)b * a.nodes;
  const float t = a.temperature ? a.temperature[b] : 1.f;
  const double s = t > 0.f ? log2_scale(t) : 0.0;
  int stop = -1;
  for (int j0 = 0; stop < 0; j0 += kChainWaves) {
    const int j = j0 + wave;
    int no = 0;
    Row r = {-INFINITY, -1, 0.0};
    if (j < a.nodes) {
      no = 1;  // the last row has no draft
      const int x = j + 1 < a.nodes ? a.tokens[at + j + 1] : -1;
      const bool draft = x >= 0 && x < a.vocab;
      const float logit = draft ? Elem<DT>::load(row_of<DT>(a, b, j)[x]) : 0.f;
      const float q = draft ? a.q[b * a.q_stride_batch + j * a.q_stride_node + x] : 0.f;
      r = row_stat<DT>(a, chunks, b, j, t);
      if (draft) no = !(fraction(a.u[at + j]) * (double)q < probability(r, t, s, x, logit));
    }
    __syncthreads();
    if (lane == 0) {
      refused[wave] = no;
      rows[wave] = r;
    }
    __syncthreads();
    for (int w = kChainWaves - 1; w >= 0; --w)
      if (refused[w]) stop = j0 + w;
  }
  const Row r = rows[stop % kChainWaves];
  const int chunk = blockIdx.x * kChainWaves + wave;
  if (blockIdx.x == 0 && threadIdx.x == 0) ends[b] = {r.z, r.top, stop, r.first};
  if (chunk >= chunks || stop + 1 == a.nodes || !(t > 0.f)) return;
  const int64_t from = (int64_t)chunk * kChunk;
  const float* q = a.q + b * a.q_stride_batch + stop * a.q_stride_node;
  const auto* row = row_of<DT>(a, b, stop);
  const double inv = r.z > 0.0 ? 1.0 / r.z : 0.0;
  double sum = 0.0;
  if (from + kChunk <= a.vocab && r.top < INFINITY) {
    constexpr int P = Elem<DT>::kPiece;
    const double m = r.top;
#pragma unroll
    for (int i = 0; i < kLane; i += P) {
      const int64_t j = place<DT>(from, a.vocab, i);
      float x[P];
      Elem<DT>::unpack(load_piece(row + j), x);
#pragma unroll
      for (int h = 0; h < P; h += 4) {
        const u32x4 v = load_piece(q + j + h);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const double y = ((double)x[h + c] - m) * s, w = pow2_or_0(y);
          const double d = w * inv - (double)bits_to_f32(v[c]);
          sum += d > 0.0 ? d : 0.0;
        }
      }
    }
  } else {
#pragma unroll 1
    for (int64_t j = from + lane; j < from + kChunk && j < a.vocab; j += 64)
      sum += residual(r, s, inv, Elem<DT>::load(row[j]), q[j]);
  }
  sum = wave_sum(sum);
  if (lane == 0) sums[(int64_t)b * chunks + chunk] = sum;
}

// One workgroup per sequence: the token after the accepted drafts.
template <int DT>
__global__ __launch_bounds__(kSampleThreads) void chain_next_kernel(VerifyArgs a, int chunks, const double* sums,
                                                                    const ChainEnd* ends) {
  __shared__ Found f;
  const int b = blockIdx.x;
  const ChainEnd end = ends[b];
  const float t = a.temperature ? a.temperature[b] : 1.f, u = a.u[(int64_t)b * a.nodes + a.nodes - 1];
  const auto* row = row_of<DT>(a, b, end.row);
  Cross at = {-1, 0.0, 0.0};
  if (end.row + 1 < a.nodes && t > 0.f) at = cross_chunk(chunks, fraction(u), [&](int c) { return sums[(int64_t)b * chunks + c]; });
  int token;
  if (!(t > 0.f)) {
    token = end.first;
  } else if (at.chunk >= 0) {
    const Row r = {end.top, end.first, end.z};
    const double s = log2_scale(t), inv = r.z > 0.0 ? 1.0 / r.z : 0.0;
    const float* q = a.q + b * a.q_stride_batch + end.row * a.q_stride_node;
    const int64_t from = (int64_t)at.chunk * kChunk + threadIdx.x * kRun;
    float x[kRun], qx[kRun];
    double w[kRun];
    load_run<DT>(row, from, a.vocab, x);
    load_run<TF_DT_F32>(q, from, a.vocab, qx);
#pragma unroll
    for (int i = 0; i < kRun; ++i) w[i] = from + i < a.vocab ? residual(r, s, inv, x[i], qx[i]) : 0.0;
    token = at.chunk * kChunk + cross_place(w, at.before, at.goal, f);
  } else {
    const ChunkStat* stat = static_cast<const ChunkStat*>(a.workspace) + ((int64_t)b * a.nodes + end.row) * chunks;
    token = sample_row<DT>(row, stat, chunks, a.vocab, t, u, f);
  }
  if (threadIdx.x == 0) {
    a.count[b] = end.row + 1;
    a.next[b] = token;
  }
}

static int chunks_of(int vocab) { return (int)(((int64_t)vocab + kChunk - 1) / kChunk); }

// The other launches of a call have fewer work-items than these, whatever its sizes.
bool verify_fits(int batch, int nodes, int vocab, bool tree) {
  const int64_t rows = (int64_t)batch * nodes;
  return launchable((rows * chunks_of(vocab) + kWaves - 1) / kWaves, kWaves * 64) && (!tree || launchable(rows, kSampleThreads));
}

template <int DT>
static hipError_t launch(const VerifyArgs& a, hipStream_t stream) {
  const int chunks = chunks_of(a.vocab);
  const int64_t rows = (int64_t)a.batch * a.nodes, groups = (rows * chunks + kWaves - 1) / kWaves;
  hipLaunchKernelGGL(chunk_kernel<DT>, dim3((unsigned)groups), dim3(kWaves * 64), 0, stream, a, chunks);
  if (a.parents != nullptr) {
    int32_t* token = reinterpret_cast<int32_t*>(static_cast<ChunkStat*>(a.workspace) + rows * chunks);
    hipLaunchKernelGGL(token_kernel<DT>, dim3((unsigned)rows), dim3(kSampleThreads), 0, stream, a, chunks, token);
    hipLaunchKernelGGL(walk_kernel, dim3(a.batch), dim3(64), 0, stream, a, token);
  } else {
    double* sums = reinterpret_cast<double*>(static_cast<ChunkStat*>(a.workspace) + rows * chunks);
    ChainEnd* ends = reinterpret_cast<ChainEnd*>(sums + (int64_t)a.batch * chunks);
    hipLaunchKernelGGL(chain_kernel<DT>, dim3((chunks + kChainWaves - 1) / kChainWaves, a.batch), dim3(kChainWaves * 64), 0, stream,
                       a, chunks, sums, ends);
    hipLaunchKernelGGL(chain_next_kernel<DT>, dim3(a.batch), dim3(kSampleThreads), 0, stream, a, chunks, sums, ends);
  }
  return hipGetLastError();
}

size_t verify_workspace(int batch, int nodes, int vocab) {
  const size_t chunks = (size_t)chunks_of(vocab), b = (size_t)(batch < 1 ? 1 : batch);
  const size_t tree = b * nodes * sizeof(int32_t), chain = b * (chunks * sizeof(double) + sizeof(ChainEnd));
  return (b * nodes * chunks * sizeof(ChunkStat) + (tree > chain ? tree : chain) + 15) / 16 * 16;
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
  if (a.dtype == TF_DT_F32) return launch<TF_DT_F32>(a, stream);
  if (a.dtype == TF_DT_F16) return launch<TF_DT_F16>(a, stream);
  return launch<TF_DT_BF16>(a, stream);
}

}  // namespace tf_exl3
