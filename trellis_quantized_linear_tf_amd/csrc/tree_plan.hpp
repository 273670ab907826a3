// What the attention kernels of drafted trees share: the line of all tiles of all sequences, heads and row
// tiles, cut into pieces of equal time on the device, and the second kernel that joins what the pieces leave.
#pragma once

#include <math.h>

#include "attention_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

// Where a sequence begins in the line, and how many tiles each of its groups has there,
// behind `start` places that stand for what it costs to begin one.
struct SeqTiles {
  int64_t begin;
  int tiles, start, piece;  // piece: places of a workgroup
};

struct AttnPlan {
  int rows, group;     // of one kv head: nodes * group
  int row_tiles;       // of one kv head
  int groups;          // kv_heads * row_tiles, each with all tiles of a sequence
  int workgroups;      // pieces, at most; 0: one for each group of each sequence
  int min_piece;       // tiles
  float c, slack;      // |scale| log2(e); the type's slack in scores
  bool negate;         // scale < 0
  uint32_t page_bytes, slot_bytes;  // of both caches, where they are the same and below 4 GiB
  int step_cols, step_slots;        // a tile in pages and slots
  FastDiv by_group, by_page, by_row_tiles, by_rows, by_groups;
  SeqTiles* seq;       // [batch]
  float2* stat;        // [2 pieces][rows of a tile] base (in log2 units), sum
  float* part;         // [2 pieces][rows of a tile][dim]
  uint32_t v_page_bytes, v_slot_bytes;  // a cache in 4 bits: of the values' cache, the ones above of the keys'
};

// The kernel's arguments, read from the argument segment where they are needed: the
// asm keeps each phase's reads in that phase, or all of them would live in scalar
// registers (and spill) from the start.
struct AttnArgs {
  tf_exl3_tree_attention_args a;
  AttnPlan p;
};
typedef const __attribute__((address_space(4))) AttnArgs* ArgPtr;
typedef const __attribute__((address_space(4))) FastDiv* DivPtr;

__device__ __forceinline__ ArgPtr arguments() {
  ArgPtr x = (ArgPtr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(x));
  return x;
}

__device__ __forceinline__ FastDiv copy(DivPtr d) { return {d->m, d->shift}; }

__device__ __forceinline__ int cached(ArgPtr x, int b) {
  const int64_t room = (int64_t)x->a.table_pages * x->a.page_size;
  const int64_t len = x->a.lengths[b];
  return (int)(len < 0 ? 0 : len > room ? room : len);
}

// n / d, of values that seldom need 64 bits.
__device__ __forceinline__ int64_t divide(int64_t n, int64_t d) {
  if (((n | d) >> 32) == 0) return (uint32_t)n / (uint32_t)d;
  return n / d;
}

// A value that all lanes have, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// A stretch of one group's places in the line.
struct Segment {
  int b, group, place, left;  // place: in the group; left: places of the piece from here on
  int len;                    // of the sequence in the cache
  int64_t begin;              // of the sequence in the line
  int start, piece;           // as in SeqTiles
  int index;                  // of the piece
};

constexpr int kMostPieces = 96;
// Tiles' worth of time to begin a group (queries, page numbers and the first tile, one behind the
// other; its rows written). With equal tiles the workgroups with two groups ended last: 64-node trees 72.8
// us against 69.1, 8 sequences of 16 nodes over 3000 positions 34.0 against 32.4.
constexpr int kStart = 4;

// Workgroups with the same number modulo this run on one XCD and share its cache.
constexpr int kTreeXCDs = 8;

// Where the workgroup's piece begins. NEAR: neighbouring pieces go to one XCD. Sequences are looked at 64 at a time, a lane each; the
// lengths of up to 64 are read once.
template <int KT, int START = kStart, bool NEAR = false>
__device__ __forceinline__ bool find_piece(ArgPtr x, int w, Segment* s) {
  const int batch = x->a.batch, groups = x->p.groups, workgroups = x->p.workgroups, nodes = x->a.nodes;
  if (workgroups == 0) {
    s->b = copy(&x->p.by_groups).div(w), s->group = w - s->b * groups;
    s->len = uniform(cached(x, s->b));
    s->place = 0, s->left = (s->len + nodes + KT - 1) / KT, s->begin = 0, s->start = s->piece = 0;
    return true;
  }
  const int lane = threadIdx.x & 63;
  int len = 0, tiles = 0;
  uint32_t end = 0;  // tiles up to and with the lane's sequence
  auto look = [&](int b0) {
    const bool there = b0 + lane < batch;
    len = there ? cached(x, b0 + lane) : 0;
    tiles = there ? (len + nodes + KT - 1) / KT : 0;
    end = (uint32_t)wave_scan(tiles);  // at most 64 times 2^30 positions in tiles of 32: 2^31
  };
  int64_t all = 0;
  for (int b0 = 0; b0 < batch; b0 += 64) {
    look(b0);
    all += (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
  }
  // Equal pieces, but no more than about kMostPieces of a row, which all have to be joined.
  const int64_t even = divide(all * groups, workgroups), joined = divide(all, (int64_t)batch * kMostPieces);
  const int start = uniform((int)(even / 4 < START ? even / 4 : START));
  all = (all + (int64_t)batch * start) * groups;
  int64_t size = divide(all + workgroups - 1, workgroups);
  size = size > joined ? size : joined;
  s->piece = uniform((int)(size < x->p.min_piece ? x->p.min_piece : size));
  s->start = start;
  if (NEAR) {
    const int used = (int)divide(all + s->piece - 1, s->piece);
    if (w >= used) return false;
    const int xcd = w % kTreeXCDs;
    w = xcd * (used / kTreeXCDs) + min(xcd, used % kTreeXCDs) + w / kTreeXCDs;
  }
  s->index = w;
  const int64_t from = (int64_t)w * s->piece;
  if (from >= all) return false;
  s->left = (int)(all - from < s->piece ? all - from : s->piece);
  int64_t base = 0;
  for (int b0 = 0;; b0 += 64) {
    if (batch > 64) look(b0);
    const uint64_t hit = __ballot((base + end + (int64_t)(lane + 1) * start) * groups > from);
    if (hit) {
      const int at = __builtin_ctzll(hit), n = __builtin_amdgcn_readlane(tiles, at) + start;
      s->b = b0 + at;
      s->len = __builtin_amdgcn_readlane(len, at);
      s->begin = (base + (uint32_t)__builtin_amdgcn_readlane((int)end, at) + (int64_t)(at + 1) * start - n) * groups;
      s->group = uniform((int)divide(from - s->begin, n));
      s->place = (int)(from - s->begin - (int64_t)s->group * n);
      return true;
    }
    base += (uint32_t)__builtin_amdgcn_readlane((int)end, 63) + 64ll * start;
  }
}

// Bits 0 .. 3: whether a row of mask `seen` sees the positions that begin `node` behind the
// cache's end (before it where negative), `left` before the run's.
__device__ __forceinline__ uint32_t seen_of(uint64_t seen, int node, int left) {
  const int before = min(-node, 4);
  const uint32_t tree = node >= 0 ? (uint32_t)(seen >> min(node, 63)) : ((uint32_t)seen << before) | ((1u << before) - 1);
  return tree & (left >= 4 ? 15u : left <= 0 ? 0u : (1u << left) - 1);
}

// WAVES waves per row: the weights of the pieces that its tiles lie in, a lane each, then their
// outputs, four columns a lane and as many pieces at a time as a wave has lanes for. Several
// waves take every WAVES-th piece each, and the first joins what they have.
template <int DT, int LANES, int WAVES>
__global__ __launch_bounds__(256) void tree_attention_join_kernel(AttnArgs args, FastDiv by_tile, int tile_rows) {
  constexpr int kSlices = 64 / LANES, kRows = 4 / WAVES;
  __shared__ f32x4 out_part[WAVES > 1 ? WAVES - 1 : 1][LANES];
  __shared__ float2 stat_part[WAVES];
  const tf_exl3_tree_attention_args& a = args.a;
  const AttnPlan& p = args.p;
  const int wave = uniform((int)threadIdx.x >> 6), sub = wave % WAVES, lane = threadIdx.x & 63;
  const int b = blockIdx.y, row = blockIdx.x * kRows + wave / WAVES;  // (head, row of it)
  if (row >= a.kv_heads * p.rows) return;
  const int g = p.by_rows.div(row), r = row - g * p.rows, tile = by_tile.div(r);
  const SeqTiles seq = p.seq[b];
  const int64_t begin = seq.begin + (int64_t)(g * p.row_tiles + tile) * (seq.tiles + seq.start);
  const int64_t from = divide(begin + seq.start, seq.piece);
  const int pieces = (int)(divide(begin + seq.start + seq.tiles - 1, seq.piece) - from) + 1;
  if (pieces == 1) return;
  // The first piece may have begun with another group; the others begin with this one.
  const int64_t head = (from * 2 + (begin > from * seq.piece)) * tile_rows + r - tile * tile_rows;
  const int64_t next = from * 2 * tile_rows + r - tile * tile_rows, step = 2 * tile_rows;
  auto at = [&](int i) { return i == 0 ? head : next + i * step; };
  const int slice = lane / LANES, d = lane % LANES * 4;
  const bool have = d < a.head_dim;
  float top = -INFINITY, z = 0.f;
  f32x4 o = f32x4(0.f);
  for (int r0 = sub; r0 < pieces; r0 += 64 * WAVES) {
    const int mine = r0 + lane * WAVES, here = min(64, (pieces - r0 + WAVES - 1) / WAVES);
    float2 st = make_float2(-INFINITY, 0.f);
    if (lane < here) st = p.stat[at(mine)];
    const float grown = fmaxf(top, wave_max(st.x));
    const float keep = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - grown);
    const float w = st.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.x - grown);
    top = grown;
    z = z * keep + wave_sum(w * st.y);
    o *= keep;
    constexpr int kAhead = 4;  // outputs on their way
    for (int i0 = 0; i0 < here; i0 += kSlices * kAhead) {  // the same for all lanes, which hold the weights
      f32x4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kSlices + slice;
        v[k] = f32x4(0.f);
        if (have && i < here) v[k] = *reinterpret_cast<const f32x4*>(p.part + at(r0 + i * WAVES) * a.head_dim + d);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kSlices + slice;
        const float wi = __builtin_bit_cast(
            float, __builtin_amdgcn_ds_bpermute((i < here ? i : 0) * 4, __builtin_bit_cast(int, w)));
        if (i < here) o += v[k] * wi;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int s = LANES; s < 64; s <<= 1) o[c] += __shfl_xor(o[c], s);
  if constexpr (WAVES > 1) {
    if (lane == 0) stat_part[sub] = make_float2(top, z);
    if (sub > 0 && slice == 0) out_part[sub - 1][lane % LANES] = o;
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const float2 st = stat_part[w];
      const float grown = fmaxf(top, st.x);
      const float mine = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - grown);
      const float its = st.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.x - grown);
      top = grown;
      z = z * mine + st.y * its;
      o = o * mine + out_part[w - 1][lane % LANES] * its;
    }
  }
  if (slice > 0 || !have) return;
  if (z == 0.f)
    o = f32x4(0.f);
  else
    o *= 1.f / z;
  const int node = p.by_group.div(r), h = g * p.group + r - node * p.group;
  uint16_t* out = static_cast<uint16_t*>(a.out) + b * a.out_stride[0] + node * a.out_stride[1] + h * a.out_stride[2] + d;
  *reinterpret_cast<u32x2*>(out) = u32x2{pack2<DT>(o[0], o[1]), pack2<DT>(o[2], o[3])};
}

// How a call's rows and positions are spread; by the sizes alone.
struct Shape {
  int dp, rt, rg, kg, kw;
  // Workgroups a CU that the line is cut for: what a CU holds at 128 columns. (At 64 the registers allow
  // twice as many, at 256 and up to 32 rows one.)
  int resident;
  int tile() const { return kg * kw; }
  int rows() const { return 16 * rt * rg; }
};

constexpr int kCUs = 256;

struct Layout {
  Shape s;
  AttnPlan p;
  size_t seq_bytes, stat_bytes, part_bytes;
  size_t workspace() const { return seq_bytes + stat_bytes + part_bytes + 16; }
};

// min_piece: tiles of a piece at least, so that writing and joining its rows costs less than its positions.
// whole(groups of all sequences): up to so many tiles a sequence, one workgroup takes all of a group's.
template <typename WHOLE>
inline Layout layout_of(const tf_exl3_tree_attention_args& a, const Shape& s, int min_piece, WHOLE whole) {
  Layout l;
  const int group = a.q_heads / a.kv_heads, rows = a.nodes * group;
  l.s = s;
  AttnPlan& p = l.p;
  p.rows = rows, p.group = group;
  p.row_tiles = (rows + l.s.rows() - 1) / l.s.rows();
  p.groups = a.kv_heads * p.row_tiles;
  p.min_piece = min_piece;
  const int64_t room = (int64_t)a.table_pages * a.page_size + a.nodes;
  const int64_t tiles = (room + l.s.tile() - 1) / l.s.tile(), most = a.batch * tiles * p.groups;
  const int64_t pieces = (most + p.min_piece - 1) / p.min_piece, slots = kCUs * l.s.resident;
  p.workgroups = (int)(pieces < slots ? pieces : slots);
  // Sequences beyond these are many enough to go one by one, and too many for every workgroup
  // to look through.
  if (a.batch > 1024 || tiles <= whole((int64_t)a.batch * p.groups)) p.workgroups = 0;
  const size_t n = (size_t)p.workgroups * 2 * l.s.rows();
  l.seq_bytes = ((size_t)a.batch * sizeof(SeqTiles) + 15) / 16 * 16;
  l.stat_bytes = (n * sizeof(float2) + 15) / 16 * 16;
  l.part_bytes = n * a.head_dim * sizeof(float);
  return l;
}

// The second launch has a workgroup for no more than each of 64 * 65535 rows, the first with pieces no more
// of them than the chip holds.
inline bool layout_fits(const tf_exl3_tree_attention_args& a, const Layout& l) {
  return launchable((int64_t)a.batch * l.p.groups, l.s.rg * l.s.kg * 64) || l.p.workgroups > 0;
}

// The rest of the plan. unit: bytes that the caches' strides count.
inline void finish_plan(const tf_exl3_tree_attention_args& a, int unit, Layout* l) {
  char* ws = static_cast<char*>(a.workspace);
  l->p.seq = reinterpret_cast<SeqTiles*>(ws);
  l->p.stat = reinterpret_cast<float2*>(ws + l->seq_bytes);
  l->p.part = reinterpret_cast<float*>(ws + l->seq_bytes + l->stat_bytes);
  // A scale of 0 keeps masked scores apart from others: the smallest factor does the same to sums.
  const float c = fabsf(a.scale) * 1.4426950408889634f;
  l->p.c = c > 1.2e-38f ? c : 1.2e-38f;
  const float slack = a.dtype == TF_DT_F16 ? Weights<TF_DT_F16>::kSlack : Weights<TF_DT_BF16>::kSlack;
  l->p.slack = fminf(slack / l->p.c, 3e38f);
  l->p.negate = a.scale < 0.f;
  const int64_t page = a.k_cache_stride[0] * unit, slot = a.k_cache_stride[1] * unit;
  const bool same = a.v_cache_stride[0] * unit == page && a.v_cache_stride[1] * unit == slot;
  l->p.page_bytes = same && page < (1ll << 32) && slot < (1ll << 32) ? (uint32_t)page : 0;
  l->p.slot_bytes = (uint32_t)slot;
  l->p.step_cols = l->s.tile() / a.page_size, l->p.step_slots = l->s.tile() % a.page_size;
  l->p.by_group = fast_div(l->p.group), l->p.by_page = fast_div(a.page_size);
  l->p.by_row_tiles = fast_div(l->p.row_tiles), l->p.by_rows = fast_div(l->p.rows), l->p.by_groups = fast_div(l->p.groups);
}

inline unsigned grid_of(const tf_exl3_tree_attention_args& a, const AttnPlan& p) {
  return p.workgroups ? (unsigned)p.workgroups : (unsigned)a.batch * (unsigned)p.groups;
}

// Joins the pieces' rows, if the line was cut.
template <int DT, int DP>
inline void launch_join(const tf_exl3_tree_attention_args& a, const AttnPlan& p, int tile_rows, hipStream_t stream) {
  if (p.workgroups == 0) return;
  const int rows = a.kv_heads * p.rows;
  const FastDiv by_tile = fast_div(tile_rows);
  if ((int64_t)rows * a.batch < kCUs * 4)  // too few rows to fill the chip with a wave each
    hipLaunchKernelGGL((tree_attention_join_kernel<DT, DP / 4, 4>), dim3(rows, a.batch), dim3(256), 0, stream,
                       AttnArgs{a, p}, by_tile, tile_rows);
  else
    hipLaunchKernelGGL((tree_attention_join_kernel<DT, DP / 4, 1>), dim3((rows + 3) / 4, a.batch), dim3(256), 0, stream,
                       AttnArgs{a, p}, by_tile, tile_rows);
}

}  // namespace tf_exl3
