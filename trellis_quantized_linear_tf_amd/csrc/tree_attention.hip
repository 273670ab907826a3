// Attention of a tree of drafted tokens over a paged cache.
//
// The rows of one kv head, (node, query head of its group), share every key. A workgroup
// takes a run of a sequence's positions (the cache's, then the nodes') for up to
// 16 RT RG of those rows, and walks it in tiles of KG KW positions that all its waves
// load together: keys and values go through registers, a tile ahead, into shared memory.
// Of its waves, RG groups share the rows and KG groups a tile's positions.
//
// Products are taken transposed, on 16x16x32 matrix instructions: S^T = K Q^T leaves a
// lane with 4 positions of one row per tile of 16, so the row's maximum is a maximum over
// registers and two lane swaps, its sum stays a lane's own to the end, and the
// probabilities are already where O^T = V^T P^T wants them: with the 32 positions of a
// step taken in the order {4g .. 4g+3, 16+4g .. 16+4g+3} for lane group g, in which V^T is
// read from shared memory by the transposing loads. Scores, statistics and outputs are
// in fp32; probabilities are rounded to the inputs' type for the second product (half a
// unit in the last place each, which the sum of fp32 probabilities does not see; `Weights` below
// says how far down fp16 holds that).
//
// All tiles of all sequences, heads and row tiles stand in one line, which the workgroups,
// as many as the chip holds at a time at 128 columns, cut into pieces of equal time, whatever the lengths are:
// every workgroup finds its piece from the lengths on the device. Where a piece ends within a
// sequence's tiles, it leaves fp32 outputs with their base and sum, and a second kernel
// joins them.
//
// Few rows a key: bound by the cache's bytes. 32 sequences of 16384 positions, 16 nodes, 32
// heads over 8 of 128, bf16: 2.14 GB in 393 us, 5.5 TB/s (keys and values two or three tiles
// ahead, 64 to 128 KB a CU; with one tile ahead 496 us). Many rows a key: 4 trees of 64 nodes, 48
// heads over 8, up to 8191 positions: 67 us, 480 TFLOP/s, 10 of them the second launch. Of the first's
// cycles matrix products take 0.24, other vector instructions 0.28, exponentials' quarter rate 0.09; the rest
// are barriers, of which one tile in shared memory needs two a tile, and waits for shared memory and loads. Taking
// one row tile's exponentials between another's products, two row tiles a wave, or
// independent workgroups of half the size measured 3 to 10% slower.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == TF_DT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Matrix products and reads of shared memory stay on their side; other work may cross.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x2 | 0x4 | 0x10); }

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == TF_DT_F16) {
    const half2_t h = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    const f32x2 f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
  }
}

// The four lane groups' values of a row (lanes l, l + 16, l + 32, l + 48), joined.
__device__ __forceinline__ float groups_max(float v) {
  u32x2 s = __builtin_amdgcn_permlane16_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  v = fmaxf(bits_to_f32(s[0]), bits_to_f32(s[1]));
  s = __builtin_amdgcn_permlane32_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  return fmaxf(bits_to_f32(s[0]), bits_to_f32(s[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
  u32x2 s = __builtin_amdgcn_permlane16_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  v = bits_to_f32(s[0]) + bits_to_f32(s[1]);
  s = __builtin_amdgcn_permlane32_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  return bits_to_f32(s[0]) + bits_to_f32(s[1]);
}

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

// A row's weights for the second product are 2^(x - base + kUp), its base at most kSlack below its
// largest score so far. bf16 has fp32's exponents. fp16 begins at 2^-14 and ends at 2^16: a base that stands
// for 2^13 keeps half a unit in the last place down to 2^-27 of the row's largest weight, and 2^-38 of that below
// (half a step of the subnormals). Slacks of 2^8, 2^4, 2^3, 2^2 and 1 with the room used up, fp16, us: 64-node trees
// 65.7 / 65.5 / 66.0 / 67.4 / 71.9, 32 x 16 nodes over 16384 positions 394 to 396 for all.
template <int DT>
struct Weights {
  static constexpr float kUp = DT == TF_DT_F16 ? 13.f : 0.f, kSlack = DT == TF_DT_F16 ? 2.f : 8.f;
};

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
};

constexpr int kMostPieces = 96;
// Tiles' worth of time to begin a group (queries, page numbers and the first tile, one behind the
// other; its rows written). With equal tiles the workgroups with two groups ended last: 64-node trees 72.8
// us against 69.1, 8 sequences of 16 nodes over 3000 positions 34.0 against 32.4.
constexpr int kStart = 4;

// Where the workgroup's piece begins. Sequences are looked at 64 at a time, a lane each; the
// lengths of up to 64 are read once.
template <int KT>
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
  const int start = uniform((int)(even / 4 < kStart ? even / 4 : kStart));
  all = (all + (int64_t)batch * start) * groups;
  int64_t size = divide(all + workgroups - 1, workgroups);
  size = size > joined ? size : joined;
  s->piece = uniform((int)(size < x->p.min_piece ? x->p.min_piece : size));
  s->start = start;
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

// Shared memory holds rows of DP elements in 16-byte chunks; chunk c of row r stands at
// c ^ (a function of r), so that neither the 16 rows x 16 bytes that a matrix operand of keys
// takes at once nor the 8 rows x 32 bytes of a transposing load meet in a bank.
template <int DP>
__device__ __forceinline__ int key_chunk(int r, int c) { return c ^ (DP == 64 ? (r >> 1) & 7 : r & 15); }
template <int DP>
__device__ __forceinline__ int value_chunk(int r, int c) { return c ^ (DP == 64 ? ((r >> 1) & 3) << 1 : (r & 7) << 1); }

// Four neighbouring columns' worth of 16-bit infinities and NaN to zero; whether any was.
template <int DT>
__device__ __forceinline__ bool drop_nonfinite(u32x4& v) {
  constexpr uint32_t top = DT == TF_DT_F16 ? 0x7C00u : 0x7F80u;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u = v[i];
    if ((u & top) == top) u &= 0xFFFF0000u, any = true;
    if ((u & top << 16) == top << 16) u &= 0xFFFFu, any = true;
    v[i] = u;
  }
  return any;
}

// Bits 0 .. 3: whether a row of mask `seen` sees the positions that begin `node` behind the
// cache's end (before it where negative), `left` before the run's.
__device__ __forceinline__ uint32_t seen_of(uint64_t seen, int node, int left) {
  const int before = min(-node, 4);
  const uint32_t tree = node >= 0 ? (uint32_t)(seen >> min(node, 63)) : ((uint32_t)seen << before) | ((1u << before) - 1);
  return tree & (left >= 4 ? 15u : left <= 0 ? 0u : (1u << left) - 1);
}

// S: tiles whose keys and values are on their way to registers. BUF: tiles in shared memory;
// with two of them a tile is put there while the one before is still in use.
template <int DT, int DP, int RT, int RG, int KG, int KW, int S, int BUF, int WAVES>
__global__ __launch_bounds__(RG * KG * 64, WAVES) void tree_attention_kernel(AttnArgs) {
  typedef uint16_t T;
  constexpr int kThreads = RG * KG * 64, KT = KG * KW, NC = DP / 8, NK = KW / 16, NB = KW / 32, ND = DP / 16, NQ = DP / 32;
  constexpr int kStep = kThreads / NC, kLoads = KT / kStep;  // rows between a thread's loads, and how many
  static_assert(KT % kStep == 0 && KW % 32 == 0, "");
  constexpr int kTile = KT * NC;
  constexpr int kJoin = KG > 1 ? (KG - 1) * RG * ND * 64 : 0;  // other key groups' outputs, one row tile at a time
  __shared__ u32x4 lds[2 * BUF * kTile > kJoin ? 2 * BUF * kTile : kJoin];
  __shared__ float2 join_stat[KG > 1 ? (KG - 1) * RG * 64 : 1];
  __shared__ uint64_t row_masks[16 * RT * RG];  // looked at in few tiles; registers are short in the widest form
  __shared__ int odd_values;

  ArgPtr x = arguments();
  Segment seg;
  if (!find_piece<KT>(x, blockIdx.x, &seg)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = wave % RG, kg = wave / RG;
  bool first = true;
  for (;;) {
    x = arguments();
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // what depends on it is worked out again and not kept over segments
    const int lane = tid & 63, lg = lane >> 4;
    const int nodes = x->a.nodes, b = seg.b;
    const int g = copy(&x->p.by_row_tiles).div(seg.group), row_tile = seg.group - g * x->p.row_tiles;
    const int len = seg.len, tiles = (len + nodes + KT - 1) / KT;
    const int last_place = min(tiles + seg.start, seg.place + seg.left);
    const int tile = max(0, seg.place - seg.start), until = last_place - seg.start;
    if (until <= 0) return;  // the piece ends before the group's first tile
    const int begin = tile * KT;
    const int stop = min(until * KT, len + nodes);  // positions of the segment: begin .. stop - 1
    const bool whole = tile == 0 && until == tiles;
    if (x->p.workgroups && seg.group == 0 && tile == 0 && tid == 0) x->p.seq[b] = {seg.begin, tiles, seg.start, seg.piece};
    if (tid == 0) odd_values = 0;

    // The rows' queries and masks.
    const int row0 = (row_tile * RG + rg) * 16 * RT;
    const bool active = row0 < x->p.rows;
    u32x4 q[RT][NQ];
    const uint64_t* masks = row_masks + rg * 16 * RT + (lane & 15);
    {
      const int rows = x->p.rows, group = x->p.group, dim = x->a.head_dim;
      const FastDiv by_group = copy(&x->p.by_group);
      const uint32_t flip = x->p.negate ? 0x80008000u : 0u;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int r = row0 + rt * 16 + (lane & 15), have = min(r, rows - 1);
        const int node = by_group.div(have), head = g * group + have - node * group;
        const T* row = static_cast<const T*>(x->a.q) + b * x->a.q_stride[0] + node * x->a.q_stride[1] + head * x->a.q_stride[2];
        if (kg == 0 && lg == 0)
          row_masks[rg * 16 * RT + rt * 16 + lane] = r < rows ? (uint64_t)x->a.mask[(int64_t)b * nodes + node] : 0;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const int d = i * 32 + lg * 8;
          q[rt][i] = u32x4(0u);
          if (r < rows && d < dim) q[rt][i] = *reinterpret_cast<const u32x4*>(row + d);
          q[rt][i] ^= flip;
        }
      }
    }

    // The loader's part: chunk `chunk` of rows tid / NC, + kStep, ...
    const int chunk = tid % NC, lrow = tid / NC;
    x = arguments();
    const float scale_c = x->p.c, slack = x->p.slack;
    const bool have = chunk * 8 < x->a.head_dim;
    const T* kc = static_cast<const T*>(x->a.k_cache) + g * x->a.k_cache_stride[2] + chunk * 8;
    const T* vc = static_cast<const T*>(x->a.v_cache) + g * x->a.v_cache_stride[2] + chunk * 8;
    const uint32_t page_bytes = x->p.page_bytes, slot_bytes = x->p.slot_bytes;  // page_bytes 0: wide or different strides
    const int32_t* table = x->a.table + b * x->a.table_stride;
    const int pages = x->a.pages, page_size = x->a.page_size;
    const int step_cols = x->p.step_cols, step_slots = x->p.step_slots;
    u32x4 kr[S][kLoads], vr[S][kLoads];
    // A row's page and slot go on by a tile at a time; rows behind the cache's end look at its
    // last page, which is there, and are not used.
    int page[kLoads] = {}, col[kLoads], slot[kLoads];
    const FastDiv by_page = copy(&x->p.by_page);
    const int last_col = len > 0 ? by_page.div(len - 1) : 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = begin + lrow + i * kStep;
      col[i] = by_page.div(j);
      slot[i] = j - col[i] * page_size;
    }
    auto look_up = [&]() {
      if (len > 0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) page[i] = *reinterpret_cast<const int32_t*>(
            reinterpret_cast<const char*>(table) + (uint32_t)min(col[i], last_col) * 4u);
      }
    };
    auto advance = [&]() {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        slot[i] += step_slots, col[i] += step_cols;
        const bool wrap = slot[i] >= page_size;
        slot[i] -= wrap ? page_size : 0, col[i] += wrap;
      }
    };
    auto load = [&](int at, u32x4 (&kr)[kLoads], u32x4 (&vr)[kLoads]) {
      const bool edge = at + KT > min(len, stop);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t pg = (uint32_t)page[i] < (uint32_t)pages ? page[i] : 0;
        const T *kp, *vp;
        if (page_bytes) {
          const uint64_t off = (uint64_t)pg * page_bytes + (uint64_t)(uint32_t)slot[i] * slot_bytes;
          kp = reinterpret_cast<const T*>(reinterpret_cast<const char*>(kc) + off);
          vp = reinterpret_cast<const T*>(reinterpret_cast<const char*>(vc) + off);
        } else {
          const ArgPtr y = arguments();
          kp = kc + pg * y->a.k_cache_stride[0] + slot[i] * y->a.k_cache_stride[1];
          vp = vc + pg * y->a.v_cache_stride[0] + slot[i] * y->a.v_cache_stride[1];
        }
        if (edge) {
          const ArgPtr y = arguments();
          const int j = at + lrow + i * kStep, node = min(j, stop - 1) - len;  // behind the run's end its last row again
          const T* kt = static_cast<const T*>(y->a.k) + b * y->a.k_stride[0] + node * y->a.k_stride[1] + g * y->a.k_stride[2];
          const T* vt = static_cast<const T*>(y->a.v) + b * y->a.v_stride[0] + node * y->a.v_stride[1] + g * y->a.v_stride[2];
          kp = j < len ? kp : kt + chunk * 8;
          vp = j < len ? vp : vt + chunk * 8;
        }
        kr[i] = *reinterpret_cast<const u32x4*>(kp);
        vr[i] = *reinterpret_cast<const u32x4*>(vp);
      }
    };

    f32x4 o[ND][RT];
    float m[RT], z[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY, z[rt] = 0.f;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) o[dt][rt] = f32x4(0.f);
    }
    const int key_row = (kg * KW + (lane & 15)) * NC;
    const int vrow = lg * 4 + ((lane & 15) >> 2);  // of the 32 positions of a step, and 16 behind
    const int value_row = kTile + (kg * KW + vrow) * NC;

    // A tile from its registers into shared memory, and the registers' next one on its way.
    auto put = [&](int at, u32x4* to, u32x4 (&kr)[kLoads], u32x4 (&vr)[kLoads]) {
      if (!have) return;
      if (at + KT > min(len, stop)) {
        // A node's values that are no numbers would reach the rows that do not see it as 0 times
        // them; they are put back below.
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int j = at + lrow + i * kStep;
          if (j >= stop) vr[i] = u32x4(0u);
          if (j >= len && drop_nonfinite<DT>(vr[i])) odd_values = 1;
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = lrow + i * kStep;
        to[r * NC + key_chunk<DP>(r, chunk)] = kr[i];
        to[kTile + r * NC + value_chunk<DP>(r, chunk)] = vr[i];
      }
      if (at + S * KT < stop) {
        load(at + S * KT, kr, vr);
        advance();
        look_up();
      }
    };
    if (have) {
      look_up();
#pragma unroll
      for (int st = 0; st < S; ++st) {
        if (begin + st * KT < stop) load(begin + st * KT, kr[st], vr[st]);
        advance();
        look_up();
      }
    } else {
      // Columns behind the head's are zero throughout.
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = lrow + i * kStep;
#pragma unroll
        for (int n = 0; n < BUF; ++n) {
          lds[2 * n * kTile + r * NC + key_chunk<DP>(r, chunk)] = u32x4(0u);
          lds[(2 * n + 1) * kTile + r * NC + value_chunk<DP>(r, chunk)] = u32x4(0u);
        }
      }
    }
    __syncthreads();
    put(begin, lds, kr[0], vr[0]);
    int half = 0;  // of shared memory, with the tile in use
    for (int at0 = begin; at0 < stop; at0 += S * KT) {
#pragma unroll
      for (int st = 0; st < S; ++st) {
        const int at = at0 + st * KT;
        if (at >= stop) break;
        const bool edge = at + KT > min(len, stop);
        __syncthreads();  // the tile is there, and with BUF 2 the one before it no longer in use
        if (active) {
          const u32x4* tile = lds + half;
          // Scores relative to the row's base m, which the products are summed onto: however large scores
          // are, those that have weight are near 0 here, and no rounding of a scaled base is in their
          // exponents (it left nothing, or infinities, from 2^23 on in fp16; 64-node trees 65.7 -> 66.1 us).
          f32x4 s[NK][RT];
#pragma unroll
          for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[t][rt] = f32x4(m[rt] == -INFINITY ? 0.f : -m[rt]);
          // Operands are read kAhead products ahead, or a product would wait out the read of its own.
          constexpr int kAhead = RT == 3 ? 1 : 2, kRing = kAhead + 1;
          u32x4 kf[kRing];
          auto key_operand = [&](int n) { return tile[key_row + n % NK * 16 * NC + key_chunk<DP>(lane & 15, n / NK * 4 + lg)]; };
#pragma unroll
          for (int n = 0; n < kAhead; ++n) kf[n] = key_operand(n);
#pragma unroll
          for (int n = 0; n < NQ * NK; ++n) {
            if (n + kAhead < NQ * NK) kf[(n + kAhead) % kRing] = key_operand(n + kAhead);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[n % NK][rt] = mfma<DT>(kf[n % kRing], q[rt][n / NK], s[n % NK][rt]);
            keep_order();
          }

          if (edge) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const uint64_t seen = masks[rt * 16];
#pragma unroll
              for (int t = 0; t < NK; ++t) {
                const int j = at + kg * KW + t * 16 + lg * 4;  // the first of the lane's four
                const uint32_t bits = seen_of(seen, j - len, stop - j);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][rt][i] = (bits >> i) & 1 ? s[t][rt][i] : -INFINITY;
              }
            }
          }

          // The base m of a row's exponents is raised, and its sums scaled, only where a score has
          // grown past it by the type's slack. Until then a lane looks at its own positions alone. (One look
          // for all row tiles cost 69.2 us against 67.4 in fp16's 64-node trees.)
          float top[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            top[rt] = s[0][rt][0];
#pragma unroll
            for (int t = 0; t < NK; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) top[rt] = fmaxf(top[rt], s[t][rt][i]);
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const bool none = m[rt] == -INFINITY;
            if (!__ballot(top[rt] > (none ? -INFINITY : slack))) continue;
            const float most = groups_max(top[rt]);
            const float up = none ? (most == -INFINITY ? 0.f : most) : fmaxf(most, 0.f);
            const float keep = none ? 0.f : __builtin_amdgcn_exp2f(-up * scale_c);
            m[rt] = none ? most : m[rt] + up;
            z[rt] *= keep;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) o[dt][rt] *= keep;
#pragma unroll
            for (int t = 0; t < NK; ++t) s[t][rt] -= up;
          }
          u32x4 pf[NB][RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < NK; ++t) {
              float e[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][rt][i], scale_c, Weights<DT>::kUp));
                sum += e[i];
              }
              pf[t / 2][rt][(t & 1) * 2] = pack2<DT>(e[0], e[1]);
              pf[t / 2][rt][(t & 1) * 2 + 1] = pack2<DT>(e[2], e[3]);
            }
            z[rt] += sum;
          }
          u32x4 vf[kRing];
          auto value_operand = [&](int n) {
            // chunks 2 dt and 2 dt + 1 of the row, 8 bytes a lane
            const u32x4* row = tile + value_row + n / ND * 32 * NC + value_chunk<DP>(vrow, n % ND * 2 + ((lane & 3) >> 1));
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(reinterpret_cast<const s16x4*>(row) + (lane & 1)));
            const s16x4 hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(reinterpret_cast<const s16x4*>(row + 16 * NC) + (lane & 1)));
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
          };
#pragma unroll
          for (int n = 0; n < kAhead; ++n) vf[n] = value_operand(n);
#pragma unroll
          for (int n = 0; n < NB * ND; ++n) {
            if (n + kAhead < NB * ND) vf[(n + kAhead) % kRing] = value_operand(n + kAhead);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) o[n % ND][rt] = mfma<DT>(vf[n % kRing], pf[n / ND][rt], o[n % ND][rt]);
            keep_order();
          }
        }
        if (at + KT < stop) {
          if (BUF == 1) __syncthreads();
          half = BUF == 1 ? 0 : 2 * kTile - half;
          put(at + KT, lds + half, kr[(st + 1) % S], vr[(st + 1) % S]);
        }
      }
    }

    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) z[rt] = groups_sum(z[rt]);
    if constexpr (KG > 1) {
      // Key group 0 takes in the others' rows, in order.
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        __syncthreads();
        if (kg > 0) {
          const int w = (kg - 1) * RG + rg;
          join_stat[w * 64 + lane] = make_float2(m[rt], z[rt]);
#pragma unroll
          for (int dt = 0; dt < ND; ++dt) lds[(w * ND + dt) * 64 + lane] = __builtin_bit_cast(u32x4, o[dt][rt]);
        }
        __syncthreads();
        if (kg == 0) {
#pragma unroll
          for (int other = 0; other < KG - 1; ++other) {
            const int w = other * RG + rg;
            const float2 st = join_stat[w * 64 + lane];
            const float top = fmaxf(m[rt], st.x);
            const float mine = m[rt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[rt] - top) * scale_c);
            const float its = st.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.x - top) * scale_c);
            m[rt] = top;
            z[rt] = z[rt] * mine + st.y * its;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt)
              o[dt][rt] = o[dt][rt] * mine + __builtin_bit_cast(f32x4, lds[(w * ND + dt) * 64 + lane]) * its;
          }
        }
      }
    }
    if (kg == 0 && active) {
      x = arguments();
      const int dim = x->a.head_dim;
      if (odd_values) {
        for (int j = max(len, begin); j < stop; ++j) {
          const T* row = static_cast<const T*>(x->a.v) + b * x->a.v_stride[0] + g * x->a.v_stride[2] + (j - len) * x->a.v_stride[1];
#pragma unroll
          for (int dt = 0; dt < ND; ++dt) {
            if (dt * 16 >= dim) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = Elem<DT>::load(row[dt * 16 + lg * 4 + i]), odd = fabsf(v) < INFINITY ? 0.f : v;
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) o[dt][rt][i] += (masks[rt * 16] >> (j - len)) & 1 ? odd : 0.f;
            }
          }
        }
      }

      const int rows = x->p.rows, group = x->p.group;
      const FastDiv by_group = copy(&x->p.by_group);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int r = row0 + rt * 16 + (lane & 15);
        if (r >= rows) continue;
        if (whole) {
          const int node = by_group.div(r), head = g * group + r - node * group;
          T* out = static_cast<T*>(x->a.out) + b * x->a.out_stride[0] + node * x->a.out_stride[1] +
                   head * x->a.out_stride[2] + lg * 4;
          const float inv = z[rt] == 0.f ? 0.f : 1.f / z[rt];
#pragma unroll
          for (int dt = 0; dt < ND; ++dt)
            if (dt * 16 < dim) {
              const f32x4 v = z[rt] == 0.f ? f32x4(0.f) : o[dt][rt] * inv;
              *reinterpret_cast<u32x2*>(out + dt * 16) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
            }
        } else {
          const int64_t row = ((int64_t)blockIdx.x * 2 + !first) * (16 * RT * RG) + r - row_tile * (16 * RT * RG);
          if (lg == 0) x->p.stat[row] = make_float2(m[rt] == -INFINITY ? -INFINITY : m[rt] * scale_c, z[rt]);
          float* part = x->p.part + row * dim + lg * 4;
#pragma unroll
          for (int dt = 0; dt < ND; ++dt)
            if (dt * 16 < dim) *reinterpret_cast<f32x4*>(part + dt * 16) = o[dt][rt];
        }
      }
    }

    seg.left -= last_place - seg.place;
    if (seg.left <= 0) return;
    seg.place = 0, first = false;
    if (++seg.group == arguments()->p.groups) {
      seg.begin += (int64_t)(tiles + seg.start) * seg.group;
      seg.group = 0, ++seg.b;
      seg.len = uniform(cached(arguments(), seg.b));
    }
    __syncthreads();
  }
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

namespace {

// How a call's rows and positions are spread; by the sizes alone.
struct Shape {
  int dp, rt, rg, kg, kw;
  // Workgroups a CU that the line is cut for: what a CU holds at 128 columns. (At 64 the registers allow
  // twice as many, at 256 and up to 32 rows one.)
  int resident;
  int tile() const { return kg * kw; }
  int rows() const { return 16 * rt * rg; }
};

Shape shape_of(int dim, int rows) {
  const int dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  // (A wave of one row group holds 32 positions at 256 columns in half its registers.)
  if (rows <= 16 && dp < 256) return {dp, 1, 1, 2, 32, 4};
  if (rows <= 32) return {dp, 1, 2, 2, 32, 2};
  if (dp == 256) return {dp, 1, 4, 1, 32, 1};
  if (rows <= 64) return {dp, 1, 4, 2, 32, 1};
  const int two = (rows + 127) / 128 * 2, three = (rows + 191) / 192 * 3;  // row tiles of 64 that are computed
  return {dp, two < three ? 2 : 3, 4, 2, 32, 1};
}

constexpr int kCUs = 256;

struct Layout {
  Shape s;
  AttnPlan p;
  size_t seq_bytes, stat_bytes, part_bytes;
};

Layout layout_of(const tf_exl3_tree_attention_args& a) {
  Layout l;
  const int group = a.q_heads / a.kv_heads, rows = a.nodes * group;
  l.s = shape_of(a.head_dim, rows);
  AttnPlan& p = l.p;
  p.rows = rows, p.group = group;
  p.row_tiles = (rows + l.s.rows() - 1) / l.s.rows();
  p.groups = a.kv_heads * p.row_tiles;
  // A piece is never so short that writing and joining its rows costs as much as its positions.
  p.min_piece = l.s.rt > 1 ? 4 : 1;
  const int64_t room = (int64_t)a.table_pages * a.page_size + a.nodes;
  const int64_t most = a.batch * ((room + l.s.tile() - 1) / l.s.tile()) * p.groups;
  const int64_t pieces = (most + p.min_piece - 1) / p.min_piece, slots = kCUs * l.s.resident;
  p.workgroups = (int)(pieces < slots ? pieces : slots);
  // Sequences beyond these are many enough to go one by one, and too many for every workgroup
  // to look through. A few tiles take one workgroup no longer than two launches take. Whole
  // against cut, us on the GPU: one sequence of 8 heads, 1 to 4 tiles 6.6 to 10.3 / 8.8 to 10.7, 6 tiles 12.9 /
  // 10.8; 16 sequences, 4 tiles 9.6 / 15.7, 8 tiles 15.3 / 18.7, 16 tiles 24.4 / 23.7; 16 of 2 heads, 8 tiles
  // 10.4 / 10.7, 12 tiles 13.4 / 11.6.
  const int64_t tiles = (room + l.s.tile() - 1) / l.s.tile();
  if (a.batch > 1024 || tiles <= 4 || (tiles <= 8 && (int64_t)a.batch * p.groups >= 32)) p.workgroups = 0;
  const size_t n = (size_t)p.workgroups * 2 * l.s.rows();
  l.seq_bytes = ((size_t)a.batch * sizeof(SeqTiles) + 15) / 16 * 16;
  l.stat_bytes = (n * sizeof(float2) + 15) / 16 * 16;
  l.part_bytes = n * a.head_dim * sizeof(float);
  return l;
}

template <int DT, int DP, int RT, int RG, int KG, int KW, int S, int BUF, int WAVES>
void launch(const tf_exl3_tree_attention_args& a, const AttnPlan& p, hipStream_t stream) {
  const unsigned grid = p.workgroups ? (unsigned)p.workgroups : (unsigned)a.batch * (unsigned)p.groups;
  hipLaunchKernelGGL((tree_attention_kernel<DT, DP, RT, RG, KG, KW, S, BUF, WAVES>), dim3(grid), dim3(RG * KG * 64), 0, stream,
                     AttnArgs{a, p});
  if (p.workgroups == 0) return;
  const int rows = a.kv_heads * p.rows, tile_rows = 16 * RT * RG;
  const FastDiv by_tile = fast_div(tile_rows);
  if ((int64_t)rows * a.batch < kCUs * 4)  // too few rows to fill the chip with a wave each
    hipLaunchKernelGGL((tree_attention_join_kernel<DT, DP / 4, 4>), dim3(rows, a.batch), dim3(256), 0, stream,
                       AttnArgs{a, p}, by_tile, tile_rows);
  else
    hipLaunchKernelGGL((tree_attention_join_kernel<DT, DP / 4, 1>), dim3((rows + 3) / 4, a.batch), dim3(256), 0, stream,
                       AttnArgs{a, p}, by_tile, tile_rows);
}

template <int DT, int DP>
void launch_dim(const tf_exl3_tree_attention_args& a, const Layout& l, hipStream_t stream) {
  const Shape& s = l.s;
  if constexpr (DP < 256) {
    if (s.rg == 1) return launch<DT, DP, 1, 1, 2, 32, 1, 1, 2>(a, l.p, stream);
    if (s.rg == 2) return launch<DT, DP, 1, 2, 2, 32, 2, 2, 2>(a, l.p, stream);
    if (s.rt == 1) return launch<DT, DP, 1, 4, 2, 32, 3, 2, 2>(a, l.p, stream);
    if (s.rt == 2) return launch<DT, DP, 2, 4, 2, 32, 1, 2, 2>(a, l.p, stream);
    return launch<DT, DP, 3, 4, 2, 32, 1, 1, 2>(a, l.p, stream);
  } else {
    if (s.rg == 2) return launch<DT, DP, 1, 2, 2, 32, 1, 1, 1>(a, l.p, stream);
    return launch<DT, DP, 1, 4, 1, 32, 1, 2, 1>(a, l.p, stream);
  }
}

template <int DT>
void launch_type(const tf_exl3_tree_attention_args& a, const Layout& l, hipStream_t stream) {
  if (l.s.dp == 64)
    launch_dim<DT, 64>(a, l, stream);
  else if (l.s.dp == 128)
    launch_dim<DT, 128>(a, l, stream);
  else
    launch_dim<DT, 256>(a, l, stream);
}

}  // namespace

size_t tree_attention_workspace(const tf_exl3_tree_attention_args& a) {
  const Layout l = layout_of(a);
  return l.seq_bytes + l.stat_bytes + l.part_bytes + 16;
}

// The second launch has a workgroup for no more than each of 64 * 65535 rows, the first with pieces no more
// of them than the chip holds.
bool tree_attention_fits(const tf_exl3_tree_attention_args& a) {
  const Layout l = layout_of(a);
  return launchable((int64_t)a.batch * l.p.groups, l.s.rg * l.s.kg * 64) || l.p.workgroups > 0;
}

hipError_t launch_tree_attention(const tf_exl3_tree_attention_args& a, hipStream_t stream) {
  Layout l = layout_of(a);
  char* ws = static_cast<char*>(a.workspace);
  l.p.seq = reinterpret_cast<SeqTiles*>(ws);
  l.p.stat = reinterpret_cast<float2*>(ws + l.seq_bytes);
  l.p.part = reinterpret_cast<float*>(ws + l.seq_bytes + l.stat_bytes);
  // A scale of 0 keeps masked scores apart from others: the smallest factor does the same to sums.
  const float c = fabsf(a.scale) * 1.4426950408889634f;
  l.p.c = c > 1.2e-38f ? c : 1.2e-38f;
  const float slack = a.dtype == TF_DT_F16 ? Weights<TF_DT_F16>::kSlack : Weights<TF_DT_BF16>::kSlack;
  l.p.slack = fminf(slack / l.p.c, 3e38f);
  l.p.negate = a.scale < 0.f;
  const int64_t page = a.k_cache_stride[0] * 2, slot = a.k_cache_stride[1] * 2;
  const bool same = a.v_cache_stride[0] * 2 == page && a.v_cache_stride[1] * 2 == slot;
  l.p.page_bytes = same && page < (1ll << 32) && slot < (1ll << 32) ? (uint32_t)page : 0;
  l.p.slot_bytes = (uint32_t)slot;
  l.p.step_cols = l.s.tile() / a.page_size, l.p.step_slots = l.s.tile() % a.page_size;
  l.p.by_group = fast_div(l.p.group), l.p.by_page = fast_div(a.page_size);
  l.p.by_row_tiles = fast_div(l.p.row_tiles), l.p.by_rows = fast_div(l.p.rows), l.p.by_groups = fast_div(l.p.groups);
  if (a.dtype == TF_DT_F16)
    launch_type<TF_DT_F16>(a, l, stream);
  else
    launch_type<TF_DT_BF16>(a, l, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
