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
#include "tree_plan.hpp"

namespace tf_exl3 {

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

namespace {

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

// A few tiles take one workgroup no longer than two launches take. Whole
// against cut, us on the GPU: one sequence of 8 heads, 1 to 4 tiles 6.6 to 10.3 / 8.8 to 10.7, 6 tiles 12.9 /
// 10.8; 16 sequences, 4 tiles 9.6 / 15.7, 8 tiles 15.3 / 18.7, 16 tiles 24.4 / 23.7; 16 of 2 heads, 8 tiles
// 10.4 / 10.7, 12 tiles 13.4 / 11.6.
Layout layout(const tf_exl3_tree_attention_args& a) {
  const Shape s = shape_of(a.head_dim, a.nodes * (a.q_heads / a.kv_heads));
  return layout_of(a, s, s.rt > 1 ? 4 : 1, [](int64_t groups) { return groups >= 32 ? 8 : 4; });
}

template <int DT, int DP, int RT, int RG, int KG, int KW, int S, int BUF, int WAVES>
void launch(const tf_exl3_tree_attention_args& a, const AttnPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((tree_attention_kernel<DT, DP, RT, RG, KG, KW, S, BUF, WAVES>), dim3(grid_of(a, p)), dim3(RG * KG * 64), 0,
                     stream, AttnArgs{a, p});
  launch_join<DT, DP>(a, p, 16 * RT * RG, stream);
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

size_t tree_attention_workspace(const tf_exl3_tree_attention_args& a) { return layout(a).workspace(); }

bool tree_attention_fits(const tf_exl3_tree_attention_args& a) { return layout_fits(a, layout(a)); }

hipError_t launch_tree_attention(const tf_exl3_tree_attention_args& a, hipStream_t stream) {
  Layout l = layout(a);
  finish_plan(a, 2, &l);
  if (a.dtype == TF_DT_F16)
    launch_type<TF_DT_F16>(a, l, stream);
  else
    launch_type<TF_DT_BF16>(a, l, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
