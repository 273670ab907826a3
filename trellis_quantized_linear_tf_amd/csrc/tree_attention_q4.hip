// Attention of a tree of drafted tokens over a paged cache in 4 bits.
//
// As over a cache of 16-bit elements, the rows of one kv head share every key, products are taken transposed
// on 16x16x32 matrix instructions, and the line of all tiles is cut into pieces of equal time. What differs is
// what bounds it: a third of the bytes, and each number has to be made of its code. So a
// tile is worked at by one wave alone, for all rows of the workgroup (up to 16 RT): the numbers are
// made once, and nothing in the loop waits for another wave. The KG waves of a workgroup take neighbouring
// runs of 32 positions.
//
// Keys need no shared memory: a lane loads neighbouring codes of one position, an eighth
// of a 16x16x32 operand each word, in an order of the head's columns that queries share (a sum over
// columns has no order). Values are made the same way and go through the wave's own part of shared
// memory, where the transposing loads turn them. Queries are read from shared memory, their registers
// being those of the outputs.
//
// 32 sequences of 16 nodes, 32 heads over 8 of 128, 16384 positions, bf16: 677 MB in 241 us (with the join's 11), 2.8
// TB/s, where the cache in 16 bits takes 393. Vector instructions bound it: 564 a wave and tile of 32 positions x 64
// rows, 272 of them the making of 8192 numbers (17 a word of 8), and 64 matrix products, at two waves a SIMD. Of its 4.7e5 cycles a
// SIMD has 3.2e5 of vector instructions and 1.3e5 of products, 0.4e5 of them at the same time: 87% busy. Priority around the products
// is worth 2%. Measured and not kept: making a
// number's code ahead between the products 270 us; a chunk order without bank conflicts in the writes of values
// (12% of the LDS's cycles) the same 238.
// By columns, 16 nodes and one: 64 162 and 101 us, 96 234 and 143, 128 248 and 154; 256 and 16 sequences 426 and 147: 64 rows
// of 256 columns are two workgroups of 32 rows, which make the same numbers, each alone on its CU.
#include "q4_device.hpp"
#include "tree_plan.hpp"

namespace tf_exl3 {

constexpr int kQ4Positions = 32;  // of a wave's tile
constexpr int kQ4Start = 2;       // tiles of KG waves that beginning a group is counted as

// The words of a row that a lane holds, and the pairs of their groups.
template <int NQ>
struct Q4Words {
  static constexpr int kPairs = NQ > 4 ? NQ / 4 : 1;
  uint32_t word[NQ], pair[kPairs];
};

template <int NQ>
__device__ __forceinline__ void load_words(const uint8_t* row, uint32_t at, uint32_t pairs, bool second, Q4Words<NQ>& x) {
  typedef uint32_t words __attribute__((ext_vector_type(NQ < 4 ? NQ : 4), aligned(4)));
  constexpr int kEach = NQ < 4 ? NQ : 4;
#pragma unroll
  for (int i = 0; i < NQ / kEach; ++i) {
    const words v = reinterpret_cast<const words*>(row + at)[i];
#pragma unroll
    for (int j = 0; j < kEach; ++j) x.word[i * kEach + j] = v[j];
  }
  x.pair[0] = *reinterpret_cast<const uint32_t*>(row + pairs);
  // A group behind the head's last: zeros.
  if constexpr (Q4Words<NQ>::kPairs == 2) x.pair[1] = second ? *reinterpret_cast<const uint32_t*>(row + pairs + 4) : 0u;
}

// A word whose numbers are worked out where they stand: those of both branches of a condition are not
// worked out, and kept, in front of it.
__device__ __forceinline__ uint32_t here(uint32_t word) {
  asm volatile("" : "+v"(word));
  return word;
}

template <int DT, int DP, int RT, int KG, int WAVES>
__global__ __launch_bounds__(KG * 64, WAVES) void tree_attention_q4_kernel(AttnArgs) {
  typedef uint16_t T;
  constexpr int KW = kQ4Positions, KT = KG * KW, kThreads = KG * 64, kRows = 16 * RT;
  constexpr int NC = DP / 8, ND = DP / 16, NQ = DP / 32;
  // Queries, then each wave's values; in the end, in their place, the waves' outputs, a row tile at a time.
  constexpr int kQueries = kRows * NC, kShared = kQueries + KG * KW * NC;
  static_assert(NQ >= 2 && ND % KG == 0 && KG * ND * 64 <= kShared, "");
  __shared__ u32x4 lds[kShared];
  __shared__ float2 join_stat[KG * 64];
  u32x4* const queries = lds;
  __shared__ uint64_t row_masks[kRows];
  __shared__ int odd_values;

  ArgPtr x = arguments();
  Segment seg;
  // Where heads of a slot lie behind one another, 80 bytes of 128 columns each, two share most of the cache's lines: with
  // neighbouring pieces on one XCD 24 sequences of 8 nodes take 43.1 us, not 46.5, 32 of 16 nodes over 16384 positions 241,
  // not 256, and 4 trees of 64 nodes, whose row tiles read the same, 75.6, not 76.8.
  if (!find_piece<KT, kQ4Start, true>(x, blockIdx.x, &seg)) return;
  const int kg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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

    // The loader's part: words lg NQ .. of the rows lane & 15 and 16 behind.
    const int dim = x->a.head_dim;
    const bool have = lg * NQ * 8 < dim;
    const uint8_t* kc = static_cast<const uint8_t*>(x->a.k_cache) + g * x->a.k_cache_stride[2];
    const uint8_t* vc = static_cast<const uint8_t*>(x->a.v_cache) + g * x->a.v_cache_stride[2];
    const bool second = (lg * NQ / 4 + 1) * kQ4Group < dim;  // of two groups
    const uint32_t k_page = x->p.page_bytes, k_slot = x->p.slot_bytes, v_page = x->p.v_page_bytes, v_slot = x->p.v_slot_bytes;
    const int32_t* table = x->a.table + b * x->a.table_stride;
    const int pages = x->a.pages, page_size = x->a.page_size;
    const int step_cols = x->p.step_cols, step_slots = x->p.step_slots;
    Q4Words<NQ> kr[2], vr[2];
    // A row's page and slot go on by a tile at a time; rows behind the cache's end look at its
    // last page, which is there, and are not used.
    int page[2] = {}, col[2], slot[2];
    const FastDiv by_page = copy(&x->p.by_page);
    const int last_col = len > 0 ? by_page.div(len - 1) : 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int j = begin + kg * KW + t * 16 + (lane & 15);
      col[t] = by_page.div(j);
      slot[t] = j - col[t] * page_size;
    }
    auto look_up = [&]() {
      if (len > 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          page[t] = *reinterpret_cast<const int32_t*>(reinterpret_cast<const char*>(table) + (uint32_t)min(col[t], last_col) * 4u);
      }
    };
    auto advance = [&]() {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        slot[t] += step_slots, col[t] += step_cols;
        const bool wrap = slot[t] >= page_size;
        slot[t] -= wrap ? page_size : 0, col[t] += wrap;
      }
    };
    auto load = [&](int l4, const uint8_t* cache, uint32_t page_bytes, uint32_t slot_bytes, Q4Words<NQ> (&r)[2]) {
      const uint32_t words = l4 * NQ * 4, pairs = dim / 2 + l4 * NQ / 4 * 4;  // places in a row
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t pg = (uint32_t)page[t] < (uint32_t)pages ? page[t] : 0;
        const uint64_t row = (uint64_t)pg * page_bytes + (uint64_t)(uint32_t)slot[t] * slot_bytes;
        if (have) load_words<NQ>(cache + row, words, pairs, second, r[t]);
      }
    };
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int w = 0; w < NQ; ++w) kr[t].word[w] = vr[t].word[w] = 0;
#pragma unroll
      for (int i = 0; i < Q4Words<NQ>::kPairs; ++i) kr[t].pair[i] = vr[t].pair[i] = 0;
    }
    // The rows' queries and masks, on their way before the cache's rows, whose pages are looked up first.
    const int row0 = row_tile * kRows;
    constexpr int kQueryLoads = (kQueries + kThreads - 1) / kThreads;
    u32x4 q_row[kQueryLoads];
    uint64_t q_mask = 0;
    {
      const int rows = x->p.rows, group = x->p.group;
      const FastDiv by_group = copy(&x->p.by_group);
#pragma unroll
      for (int n = 0; n < kQueryLoads; ++n) {
        const int i = tid + n * kThreads, r = row0 + i / NC, c = i % NC, r_have = min(r, rows - 1);
        const int node = by_group.div(r_have), head = g * group + r_have - node * group;
        const T* row = static_cast<const T*>(x->a.q) + b * x->a.q_stride[0] + node * x->a.q_stride[1] + head * x->a.q_stride[2];
        q_row[n] = u32x4(0u);
        if (r < rows && c * 8 < dim) q_row[n] = *reinterpret_cast<const u32x4*>(row + c * 8);
      }
      if (tid < kRows && row0 + tid < rows) q_mask = (uint64_t)x->a.mask[(int64_t)b * nodes + by_group.div(row0 + tid)];
    }
    const int mine = begin + kg * KW;  // the wave's first position
    if (mine < stop) {
      look_up();
      load(lg, kc, k_page, k_slot, kr);
      load(lg, vc, v_page, v_slot, vr);
      advance();
      look_up();
    }

    {
      const uint32_t flip = x->p.negate ? 0x80008000u : 0u;
#pragma unroll
      for (int n = 0; n < kQueryLoads; ++n) {
        const int i = tid + n * kThreads, r = i / NC;
        if (kQueries % kThreads == 0 || i < kQueries) queries[r * NC + key_chunk<DP>(r, i % NC)] = q_row[n] ^ flip;
      }
      if (tid < kRows) row_masks[tid] = q_mask;
    }
    x = arguments();
    const float scale_c = x->p.c, slack = x->p.slack;

    f32x4 o[ND][RT];
    float m[RT], z[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY, z[rt] = 0.f;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) o[dt][rt] = f32x4(0.f);
    }
    u32x4* const values = lds + kQueries + kg * KW * NC;
    // Other instructions stay on their side of it: all of a tile's numbers made at once need more registers than there are.
    auto phase = []() { __builtin_amdgcn_sched_barrier(0); };
    auto in_order = [&]() {  // of the wave's own writes and reads of shared memory, for the compiler; the hardware keeps it
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      phase();
    };
    __syncthreads();

    for (int at = mine; at < stop; at += KT) {
      const bool edge = at + KW > min(len, stop), more = at + KT < stop;
      int l = lane;
      asm volatile("" : "+v"(l));  // places in shared memory are worked out again for each tile
      const int l15 = l & 15, l4 = l >> 4;
      // Numbers of a tile's keys or values into the wave's part of shared memory.
      auto fill = [&](bool value, const Q4Words<NQ> (&words)[2]) {
        in_order();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int r = t * 16 + l15;
#pragma unroll
          for (int w = 0; w < NQ; ++w) {
            values[r * NC + value_chunk<DP>(r, l4 * NQ + w)] = q4_piece<DT>(value ? words[t].word[w] : here(words[t].word[w]), words[t].pair[w / 4]);
            if (w % 2) phase();
          }
        }
        if (edge) {
          // The nodes' own rows over what lies behind the cache's end there, and zeros behind the run's end.
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int r = t * 16 + l15, node = at + r - len;
            if (node < 0) continue;
            const ArgPtr y = arguments();
            const T* row = value ? static_cast<const T*>(y->a.v) + b * y->a.v_stride[0] + node * y->a.v_stride[1] + g * y->a.v_stride[2]
                                 : static_cast<const T*>(y->a.k) + b * y->a.k_stride[0] + node * y->a.k_stride[1] + g * y->a.k_stride[2];
            u32x4 e[NQ];
            int columns = at + r < stop ? dim : 0;
            asm volatile("" : "+v"(columns));  // compared here, not kept compared for every word
#pragma unroll
            for (int w = 0; w < NQ; ++w) {
              const int c = l4 * NQ + w;
              e[w] = u32x4(0u);
              if (c * 8 < columns) e[w] = *reinterpret_cast<const u32x4*>(row + c * 8);
            }
#pragma unroll
            for (int w = 0; w < NQ; ++w) {
              // A value that is no number would reach the rows that do not see it as 0 times it; it is put back below.
              if (value && drop_nonfinite<DT>(e[w])) odd_values = 1;
              values[r * NC + value_chunk<DP>(r, l4 * NQ + w)] = e[w];
            }
          }
        }
        in_order();
      };

      // Scores relative to the row's base m, which the products are summed onto: however large scores
      // are, those that have weight are near 0 here.
      f32x4 s[2][RT];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[t][rt] = f32x4(m[rt] == -INFINITY ? 0.f : -m[rt]);
      auto query_operand = [&](int w, int rt) { return queries[(rt * 16 + l15) * NC + key_chunk<DP>(l15, l4 * NQ + w)]; };
      if (!edge) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int w = 0; w < NQ; ++w) {
          const u32x4 k0 = q4_piece<DT>(kr[0].word[w], kr[0].pair[w / 4]);
          const u32x4 k1 = q4_piece<DT>(kr[1].word[w], kr[1].pair[w / 4]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const u32x4 q = query_operand(w, rt);
            s[0][rt] = mfma<DT>(k0, q, s[0][rt]);
            s[1][rt] = mfma<DT>(k1, q, s[1][rt]);
          }
          if (w % 2) phase();
        }
        __builtin_amdgcn_s_setprio(0);
      } else {
        fill(false, kr);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int w = 0; w < NQ; ++w) {
            const u32x4 k = values[(t * 16 + l15) * NC + value_chunk<DP>(l15, l4 * NQ + w)];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[t][rt] = mfma<DT>(k, query_operand(w, rt), s[t][rt]);
            phase();
          }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint64_t seen = row_masks[rt * 16 + l15];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int j = at + t * 16 + l4 * 4;  // the first of the lane's four
            const uint32_t bits = seen_of(seen, j - len, stop - j);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][rt][i] = (bits >> i) & 1 ? s[t][rt][i] : -INFINITY;
          }
          phase();
        }
      }
      if (more) load(l4, kc, k_page, k_slot, kr);
      fill(true, vr);
      if (more) {
        load(l4, vc, v_page, v_slot, vr);
        advance();
        look_up();
      }
      phase();

      // The base of a row's exponents is raised, and its sums scaled, only where a score has grown past it by the
      // type's slack.
      u32x4 pf[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = s[0][rt][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][rt][i]);
        const bool none = m[rt] == -INFINITY;
        if (__ballot(top > (none ? -INFINITY : slack))) {
          const float most = groups_max(top);
          const float up = none ? (most == -INFINITY ? 0.f : most) : most > slack ? most : 0.f;
          const float keep = none ? 0.f : __builtin_amdgcn_exp2f(-up * scale_c);
          m[rt] = none ? most : m[rt] + up;
          z[rt] *= keep;
#pragma unroll
          for (int dt = 0; dt < ND; ++dt) o[dt][rt] *= keep;
#pragma unroll
          for (int t = 0; t < 2; ++t) s[t][rt] -= up;
        }
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][rt][i], scale_c, Weights<DT>::kUp));
            sum += e[i];
          }
          pf[rt][t * 2] = pack2<DT>(e[0], e[1]);
          pf[rt][t * 2 + 1] = pack2<DT>(e[2], e[3]);
        }
        z[rt] += sum;
        phase();
      }

      const int vrow = l4 * 4 + (l15 >> 2);  // of the 32 positions, and 16 behind
      constexpr int kAhead = 2, kRing = kAhead + 1;
      u32x4 vf[kRing];
      auto value_operand = [&](int dt) {
        // chunks 2 dt and 2 dt + 1 of the row, 8 bytes a lane
        const u32x4* row = values + vrow * NC + value_chunk<DP>(vrow, dt * 2 + ((l & 3) >> 1));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(reinterpret_cast<const s16x4*>(row) + (l & 1)));
        const s16x4 hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(reinterpret_cast<const s16x4*>(row + 16 * NC) + (l & 1)));
        return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      };
#pragma unroll
      for (int n = 0; n < kAhead; ++n) vf[n] = value_operand(n);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int n = 0; n < ND; ++n) {
        if (n + kAhead < ND) vf[(n + kAhead) % kRing] = value_operand(n + kAhead);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) o[n][rt] = mfma<DT>(vf[n % kRing], pf[rt], o[n][rt]);
        keep_order();
      }
      __builtin_amdgcn_s_setprio(0);
    }

    // The waves' rows, a row tile at a time: each wave joins a part of the columns, in the waves' order, and leaves
    // it where it belongs.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      constexpr int kMine = ND / KG;
      const float sum = groups_sum(z[rt]);
      __syncthreads();  // what was there before is no longer in use
      join_stat[kg * 64 + lane] = make_float2(m[rt], sum);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) lds[(kg * ND + dt) * 64 + lane] = __builtin_bit_cast(u32x4, o[dt][rt]);
      __syncthreads();
      float base = -INFINITY, total = 0.f;
      f32x4 own[kMine];
#pragma unroll
      for (int n = 0; n < kMine; ++n) own[n] = f32x4(0.f);
#pragma unroll
      for (int w = 0; w < KG; ++w) base = fmaxf(base, join_stat[w * 64 + lane].x);
#pragma unroll
      for (int w = 0; w < KG; ++w) {
        const float2 st = join_stat[w * 64 + lane];
        const float its = st.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.x - base) * scale_c);
        total += st.y * its;
#pragma unroll
        for (int n = 0; n < kMine; ++n) own[n] += __builtin_bit_cast(f32x4, lds[(w * ND + kg * kMine + n) * 64 + lane]) * its;
      }
      const ArgPtr y = arguments();
      const int column = kg * kMine * 16 + lg * 4;  // and 16 behind for each n
      if (odd_values) {
        const uint64_t seen = row_masks[rt * 16 + (lane & 15)];
        for (int j = max(len, begin); j < stop; ++j) {
          const T* row = static_cast<const T*>(y->a.v) + b * y->a.v_stride[0] + g * y->a.v_stride[2] + (j - len) * y->a.v_stride[1];
#pragma unroll
          for (int n = 0; n < kMine; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (column + n * 16 >= dim) continue;
              const float v = Elem<DT>::load(row[column + n * 16 + i]);
              own[n][i] += ((seen >> (j - len)) & 1) && !(fabsf(v) < INFINITY) ? v : 0.f;
            }
        }
      }
      const int r = row0 + rt * 16 + (lane & 15), group = y->p.group;
      if (r < y->p.rows) {
        if (whole) {
          const int node = copy(&y->p.by_group).div(r), head = g * group + r - node * group;
          T* out = static_cast<T*>(y->a.out) + b * y->a.out_stride[0] + node * y->a.out_stride[1] + head * y->a.out_stride[2] + column;
          const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
          for (int n = 0; n < kMine; ++n)
            if (column + n * 16 < dim) {
              const f32x4 v = total == 0.f ? f32x4(0.f) : own[n] * inv;
              *reinterpret_cast<u32x2*>(out + n * 16) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
            }
        } else {
          const int64_t row = ((int64_t)seg.index * 2 + !first) * kRows + r - row0;
          if (kg == 0 && lg == 0) y->p.stat[row] = make_float2(base == -INFINITY ? -INFINITY : base * scale_c, total);
          float* part = y->p.part + row * dim + column;
#pragma unroll
          for (int n = 0; n < kMine; ++n)
            if (column + n * 16 < dim) *reinterpret_cast<f32x4*>(part + n * 16) = own[n];
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

namespace {

// Waves a SIMD by the row tiles whose outputs a wave holds; a workgroup has four waves, so as many workgroups a CU.
constexpr int waves_of(int dp, int rt) { return dp == 256 || rt == 4 ? 2 : dp * rt == 256 ? 3 : 4; }

// Row tiles of a wave: as many as there are, up to four (two at 256 columns), as long as enough tiles are left
// to give every workgroup that the chip holds a few: a number is made once for all of a wave's rows, but one wave alone
// takes long over many rows. One, two, four row tiles, us on the GPU, 8 heads of 128, by places (tiles of 128
// positions of each row tile): 32 rows, 64 places of two row tiles 13.3 / 14.4, 1056 21.4 / 27.8, 2112 28.3 / 29.1, 6336
// 62 / 42; 64 rows, 128 places of four 15 / 16 / 19, 1024 29 / 27 / 31, 2176 44 / 35 / 38, 3968 63 / 47 / 45, 7936
// 130 / 83 / 63.
Shape shape_of(const tf_exl3_tree_attention_args& a) {
  const int dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256, rows = a.nodes * (a.q_heads / a.kv_heads);
  const int64_t tiles = ((int64_t)a.table_pages * a.page_size + a.nodes) / (4 * kQ4Positions) + 1;
  const int64_t groups = (int64_t)a.batch * a.kv_heads * tiles;
  int rt = 1;
  if (rows > 16 && groups * ((rows + 31) / 32) >= 2048) rt = 2;
  if (dp < 256 && rows > 32 && groups * ((rows + 63) / 64) >= 3200) rt = 4;
  // Workgroups a CU that the line is cut for: what it holds (of 256 columns and two row tiles, 84 KB of shared memory,
  // one), but two where a piece would be a few tiles: beginning and joining it takes as long. Two, three, four, us on the
  // GPU, 8 heads of 128: 1088 places 18.1 / 16.0 / 15.7, 1632 19.2 / 20.0 / 18.2, 1904 21.7 / 21.3 / 21.7, 2176 22.0 / 22.3 / 22.5,
  // 4608 29.0 / 31.7 / 32.9, 6240 in two row tiles 42.1 / 45.1 / -, 6336 so 41.6 / 46.4 / -, 8448 40.5 / 43.4 / 43.9, 9216 43.4 /
  // 48.8 / 47.2, 10752 49.5 / 49.7 / 53.4, 12480 65.8 / 68.5 / 63.8, 33024 154 / 150 / 151. In between it costs up to 4% elsewhere: 2 heads, 9216
  // 42.4 / 40.5 / 42.1; 16 heads 48 / 49 / 46; 1 head 2176 21.9 / 23.0 / 22.8, 9216 38.2 / 37.9 / 38.4. 64 columns: 1088 15.3 / 13.4 / 13.3, 2056
  // 27.0 / 31.2 / 31.0, 4608 22.9 / 23.8 / 24.3, 8320 29.8 / 31.5 / 32.3, 9216 31.1 / 35.4 / 33.0 (a head's slots behind one another: 22.8 /
  // 25.3 / 25.3, 20.9 / 22.0 / 22.0, 26.4 / 26.1 / 27.6, 27.5 / 27.6 / 27.2), 12480 50.2 / 50.6 / 46.6, 33024 so 105 / 95 / 93.
  const int64_t places = groups * ((rows + 16 * rt - 1) / (16 * rt));
  int resident = dp == 256 && rt == 2 ? 1 : waves_of(dp, rt);
  if (resident > 2 && places >= 2048 && places < 10240) resident = 2;
  return {dp, rt, 1, 4, kQ4Positions, resident};
}

// By the table's room, not the lengths, which are on the device: 24 sequences of 100 positions and 16 nodes take 13.5 us with a table of
// their own size and 28.6 with one for 4096 positions or more, one such sequence 8.5 and 11.2 (12.7 for 32768).
// The more groups there are, the longer one workgroup may take over one of them before two launches and pieces of
// equal time take less. Whole against cut, us on the GPU, 8 rows of 128 (32 rows): 8 groups, 3 tiles 9.9 / 11.3 (10.2 /
// 11.7), 4 tiles 11.3 / 11.4, 5 tiles 12.7 / 11.4 (13.0 / 11.8); 128 groups, 6 tiles 16.9 / 16.1 (19.6 / 23.8), 8 tiles
// 20.0 / 16.6 (23.0 / 26.9), 10 tiles 23.5 / 21.1 (26.2 / 26.1); 256 groups, 10 tiles 27.2 / 27.0 (30.1 / 33.2), 12 tiles
// 30.3 / 28.1 (32.8 / 33.8), 16 tiles 37 / 32 (41 / 36); 512 groups, 12 tiles 41 / 41 (44 / 53), 16 tiles 51 / 50 (56 /
// 56), 23 tiles 66 / 60 (76 / 81).
Layout layout(const tf_exl3_tree_attention_args& a) {
  const Shape s = shape_of(a);
  return layout_of(a, s, s.rt > 2 ? 2 : 1, [](int64_t groups) { return groups >= 512 ? 16 : groups >= 256 ? 12 : groups >= 128 ? 8 : 4; });
}

template <int DT, int DP, int RT>
void launch(const tf_exl3_tree_attention_args& a, const AttnPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((tree_attention_q4_kernel<DT, DP, RT, 4, waves_of(DP, RT)>), dim3(grid_of(a, p)), dim3(256), 0, stream,
                     AttnArgs{a, p});
  launch_join<DT, DP>(a, p, 16 * RT, stream);
}

template <int DT, int DP>
void launch_dim(const tf_exl3_tree_attention_args& a, const Layout& l, hipStream_t stream) {
  if (l.s.rt == 1) return launch<DT, DP, 1>(a, l.p, stream);
  if (l.s.rt == 2) return launch<DT, DP, 2>(a, l.p, stream);
  if constexpr (DP < 256) launch<DT, DP, 4>(a, l.p, stream);
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

size_t tree_attention_q4_workspace(const tf_exl3_tree_attention_args& a) { return layout(a).workspace(); }

bool tree_attention_q4_fits(const tf_exl3_tree_attention_args& a) { return layout_fits(a, layout(a)); }

hipError_t launch_tree_attention_q4(const tf_exl3_tree_attention_args& a, hipStream_t stream) {
  Layout l = layout(a);
  finish_plan(a, 1, &l);
  l.p.page_bytes = (uint32_t)a.k_cache_stride[0], l.p.slot_bytes = (uint32_t)a.k_cache_stride[1];
  l.p.v_page_bytes = (uint32_t)a.v_cache_stride[0], l.p.v_slot_bytes = (uint32_t)a.v_cache_stride[1];
  if (a.dtype == TF_DT_F16)
    launch_type<TF_DT_F16>(a, l, stream);
  else
    launch_type<TF_DT_BF16>(a, l, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
