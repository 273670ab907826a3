// Causal attention of whole prompts, packed behind one another.
//
// A workgroup takes a tile of kRows consecutive tokens of one query head, whatever sequences they
// belong to: each row knows where its sequence begins, and sees the keys from there to itself. So short
// sequences share a tile, and nothing has to be known of them on the host. The keys from the first row's
// beginning to the last row are walked in tiles of KT that all waves load together, straight into shared
// memory, one tile ahead; each of the four waves holds 16 RT rows.
//
// Products are transposed as in tree attention: S^T = K Q^T leaves a lane with 4 positions of one row
// per tile of 16, and its weights are where O^T = V^T P^T wants them. Only tiles that some row of a wave does
// not see as a whole are masked.
//
// One prompt of 16384 tokens, 32 heads over 8 of 128, bf16: 2.2 TFLOP in 2.00 to 2.07 ms, 1.06 to 1.10 PFLOP/s, where torch's
// product of 8192^3 reached 1.21 to 1.34 on the same cards. By the counters a wave and 64 keys take 64 matrix products and 221
// other vector instructions, 32 of them exponentials, which count twice: of a SIMD's 4.1e6 cycles the matrix core is busy for 2.1e6 and
// other vector instructions for 2.1e6, 0.5e6 of them at the same time. Steps of 32 keys whose weights are made between
// the products of the next step's scores measured 2.11 ms against 2.00. 24 prompts of 512 to 2050 tokens, fp16: 555 to 580 us,
// 640 to 660 TFLOP/s (passes under a kernel trace 583 to 628 us); a tenth of the products each are the diagonal's and those of tiles with two
// sequences' rows, and with their masks a step has 338 other vector instructions; the rest are starts and the last workgroups.
// 8 such prompts of 2048 tokens, TFLOP/s by columns, and one of 16384: 64 554 and 921, 96 536 and 852 (a quarter of the products
// are with zeros), 128 700 and 1067, 256 592 and 808 (one row tile a wave: half of the products an operand read).
#include <math.h>

#include "attention_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

struct PromptPlan {
  int tiles;           // of tokens
  int spread;          // heads of an XCD, where all of them have equally many; else 0
  float c, slack;      // |scale| log2(e); the type's slack in scores
  bool negate;         // scale < 0
  FastDiv by_heads, by_group;  // by_heads: spread, or q_heads
};

constexpr int kPromptWaves = 4, kPromptThreads = 64 * kPromptWaves;
constexpr int kXCDs = 8;
constexpr int kNowhere = 0x7FFFFFFF;  // the beginning of a row that belongs to no sequence

// Where the sequence of token i begins; kNowhere in front of the first and behind the last one.
// `sample` is a lane's entry of the wave's 64 evenly spread offsets, `every` entries apart: with 63 sequences or
// fewer they are all of them, and nothing else is loaded.
__device__ __forceinline__ int sequence_begin(const int32_t* offsets, int batch, int i, int sample, int every) {
  int lo = -1, hi = batch / every + 1;  // samples: that of lo is at most i, that of hi more, as if there were such ends
  for (int width = hi - lo; width > 1; width = (width + 1) / 2) {  // as often for every lane
    const int mid = lo + (hi - lo) / 2, v = __builtin_amdgcn_ds_bpermute(max(mid, 0) * 4, sample);
    if (hi - lo > 1) {
      if (v <= i)
        lo = mid;
      else
        hi = mid;
    }
  }
  int begin = __builtin_amdgcn_ds_bpermute(max(lo, 0) * 4, sample);
  if (lo < 0) return kNowhere;
  lo *= every, hi = min(hi * every, batch + 1);
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2, v = offsets[mid];
    if (v <= i)
      lo = mid, begin = v;
    else
      hi = mid;
  }
  return lo == batch ? kNowhere : max(begin, 0);
}

template <typename F>
__device__ __forceinline__ int rows_reduce(int v, F f) {  // over the 16 rows that a lane group holds
#pragma unroll
  for (int s = 1; s < 16; s <<= 1) v = f(v, __shfl_xor(v, s));
  return v;
}

// Whether one of the 16-bit elements of a 16-byte piece is no finite number.
template <int DT>
__device__ __forceinline__ uint32_t largest_exponents(u32x4 v, uint32_t so_far) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = v[i] & 0x7FFF7FFFu;
    so_far = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, u), __builtin_bit_cast(u16x2, so_far)));
  }
  return so_far;
}

// 16 bytes a lane, `offset` bytes from `base`, to shared memory at `to` + 16 lane (base and `to` the same
// for all lanes). The load is not among those that the compiler counts: it is waited for with wait_loads before
// the barrier behind which its bytes are read. (With the compiler's builtin every read of shared memory, of the
// other half too, waited for the loads in flight.)
__device__ __forceinline__ void load_to_shared(const void* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(to), "v"(offset), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <int DT, int DP, int RT, int KT>
__global__ __launch_bounds__(kPromptThreads, 2) void prompt_attention_kernel(tf_exl3_prompt_attention_args a, PromptPlan p) {
  typedef uint16_t T;
  constexpr int NC = DP / 8, NK = KT / 16, NB = KT / 32, ND = DP / 16, NQ = DP / 32, kRows = 16 * RT * kPromptWaves;
  constexpr int kTile = KT * NC, kStep = kPromptThreads / NC, kLoads = KT / kStep;
  static_assert(KT % kStep == 0 && KT % 32 == 0, "");
  __shared__ u32x4 lds[4 * kTile];  // keys and values of two tiles
  __shared__ int ranges[2][kPromptWaves];

  // The last tiles, which see most, come first; the heads of a kv head stay on one XCD where they can.
  int tile, head;
  {
    const int id = blockIdx.x;
    if (p.spread) {
      const int slot = id / kXCDs, t = p.by_heads.div(slot);
      tile = p.tiles - 1 - t, head = id % kXCDs * p.spread + slot - t * p.spread;
    } else {
      const int t = p.by_heads.div(id);
      tile = p.tiles - 1 - t, head = id - t * a.q_heads;
    }
  }
  const int g = p.by_group.div(head);
  const int tid = threadIdx.x, lane = tid & 63, lg = lane >> 4, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row0 = tile * kRows + wave * 16 * RT;  // the wave's first token

  const int every = a.batch / 64 + 1;
  const int sample = a.offsets[min(lane * every, a.batch)];
  u32x4 q[RT][NQ];
  {
    const uint32_t flip = p.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int i = row0 + rt * 16 + (lane & 15);
      const T* row = static_cast<const T*>(a.q) + i * a.q_stride[0] + head * a.q_stride[1];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int d = n * 32 + lg * 8;
        q[rt][n] = u32x4(0u);
        if (i < a.tokens && d < a.head_dim) q[rt][n] = *reinterpret_cast<const u32x4*>(row + d);
        q[rt][n] ^= flip;
      }
    }
  }
  // Rows, the beginnings of their sequences, and what the wave and the workgroup look at.
  int begin[RT];
  int low = kNowhere, high = 0, latest = 0;  // first key, past the last, latest beginning
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int i = row0 + rt * 16 + (lane & 15);
    begin[rt] = sequence_begin(a.offsets, a.batch, i, sample, every);
    if (i >= a.tokens || begin[rt] > i) begin[rt] = kNowhere;
    low = min(low, begin[rt]), latest = max(latest, begin[rt]);
    if (begin[rt] != kNowhere) high = max(high, i + 1);
  }
  low = __builtin_amdgcn_readfirstlane(rows_reduce(low, [](int x, int y) { return min(x, y); }));
  high = __builtin_amdgcn_readfirstlane(rows_reduce(high, [](int x, int y) { return max(x, y); }));
  latest = __builtin_amdgcn_readfirstlane(rows_reduce(latest, [](int x, int y) { return max(x, y); }));
  if (lane == 0) ranges[0][wave] = low, ranges[1][wave] = high;

  // Columns behind the head's are zero throughout.
  if (a.head_dim < DP) {
    for (int i = tid; i < 4 * kTile; i += kPromptThreads) lds[i] = u32x4(0u);
  }
  __syncthreads();
  int from = ranges[0][0], to = ranges[1][0];
#pragma unroll
  for (int w = 1; w < kPromptWaves; ++w) from = min(from, ranges[0][w]), to = max(to, ranges[1][w]);
  from = __builtin_amdgcn_readfirstlane(from), to = __builtin_amdgcn_readfirstlane(to);
  if (from >= to) return;

  const T* const kb = static_cast<const T*>(a.k) + g * a.k_stride[1];
  const T* const vb = static_cast<const T*>(a.v) + g * a.v_stride[1];
  // The loader's part: chunk tid % NC of rows tid / NC, + kStep, ... as shared memory has them. Of 8 rows
  // between them (256 columns) two neighbours differ in the place of a key's chunk.
  constexpr int kKinds = kStep < 16 ? 2 : 1;
  const int chunk = tid % NC, lrow = tid / NC;
  const uint32_t ks = (uint32_t)a.k_stride[0] * 2, vs = (uint32_t)a.v_stride[0] * 2;  // bytes, at most 2^24
  const uint32_t place = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) u32x4*)lds + wave * 1024;
  int kc[kKinds];
#pragma unroll
  for (int n = 0; n < kKinds; ++n) kc[n] = key_chunk<DP>(lrow + n * kStep, chunk);
  const int vc = value_chunk<DP>(lrow, chunk);
  auto stage = [&](int at, int buffer) {
    const uint32_t dst = place + buffer * 2 * kTile * 16;
    const char* const kt = reinterpret_cast<const char*>(kb) + (uint64_t)(uint32_t)at * ks;
    const char* const vt = reinterpret_cast<const char*>(vb) + (uint64_t)(uint32_t)at * vs;
    const uint32_t last = min(a.tokens - 1 - at, KT);  // behind the last token its row again
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int c = kc[n % kKinds];
      const uint32_t k = min(lrow * ks + (uint32_t)(n * kStep) * ks, last * ks), v = min(lrow * vs + (uint32_t)(n * kStep) * vs, last * vs);
      if (c * 8 < a.head_dim) load_to_shared(kt, k + c * 16, dst + n * kPromptThreads * 16);
      if (vc * 8 < a.head_dim) load_to_shared(vt, v + vc * 16, dst + (kTile + n * kPromptThreads) * 16);
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
  const int key_row = (lane & 15) * NC;
  const int vrow = lg * 4 + ((lane & 15) >> 2);  // of the 32 positions of a step, and 16 behind
  const int value_row = kTile + vrow * NC;

  stage(from, 0);
  int half = 0;
  for (int at = from; at < to; at += KT) {
    wait_loads();     // this wave's part of the tile is there,
    __syncthreads();  // and everyone's; the tile before is no longer in use
    if (at + KT < to) stage(at + KT, half ^ 1);
    if (at < high && at + KT > low) {
      const u32x4* tile = lds + half * 2 * kTile;
      const bool edge = at < latest || at + KT - 1 > row0;
      // Scores relative to the row's base m, which the products are summed onto.
      f32x4 s[NK][RT];
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[t][rt] = f32x4(m[rt] == -INFINITY ? 0.f : -m[rt]);
      constexpr int kAhead = 2, kRing = kAhead + 1;
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
          // j is seen where begin <= j <= i: j - begin, as a number without a sign, is at most i - begin
          const uint32_t span = begin[rt] == kNowhere ? 0u : (uint32_t)(row0 + rt * 16 + (lane & 15) - begin[rt]);
#pragma unroll
          for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t j = (uint32_t)(at + t * 16 + lg * 4 + i - begin[rt]);
              s[t][rt][i] = j <= span ? s[t][rt][i] : -INFINITY;
            }
        }
      }

      // A row's base is raised only where one of its scores has grown past it by the type's slack, whatever
      // the other rows of the wave do.
      u32x4 pf[NB][RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = s[0][rt][0];
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][rt][i]);
        const bool none = m[rt] == -INFINITY;
        if (__ballot(top > (none ? -INFINITY : p.slack))) {
          const float most = groups_max(top);
          const float up = none ? (most == -INFINITY ? 0.f : most) : most > p.slack ? most : 0.f;
          const float keep = none ? 0.f : __builtin_amdgcn_exp2f(-up * p.c);
          m[rt] = none ? most : m[rt] + up;
          z[rt] *= keep;
#pragma unroll
          for (int dt = 0; dt < ND; ++dt) o[dt][rt] *= keep;
#pragma unroll
          for (int t = 0; t < NK; ++t) s[t][rt] -= up;
        }
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < NK; ++t) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][rt][i], p.c, Weights<DT>::kUp));
            sum += e[i];
          }
          pf[t / 2][rt][(t & 1) * 2] = pack2<DT>(e[0], e[1]);
          pf[t / 2][rt][(t & 1) * 2 + 1] = pack2<DT>(e[2], e[3]);
        }
        z[rt] += sum;
      }

      auto value_operand = [&](int n) {
        // chunks 2 dt and 2 dt + 1 of the row, 8 bytes a lane
        const u32x4* row = tile + value_row + n / ND * 32 * NC + value_chunk<DP>(vrow, n % ND * 2 + ((lane & 3) >> 1));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(reinterpret_cast<const s16x4*>(row) + (lane & 1)));
        const s16x4 hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(reinterpret_cast<const s16x4*>(row + 16 * NC) + (lane & 1)));
        return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      };
      // A value that is no finite number would reach the rows that do not see it as 0 times it.
      bool odd = false;
      if (edge) {
        uint32_t most = 0;
#pragma unroll
        for (int n = 0; n < NB * ND; ++n) most = largest_exponents<DT>(value_operand(n), most);
        constexpr uint32_t top = DT == TF_DT_F16 ? 0x7C00u : 0x7F80u;
        odd = __ballot((most & 0xFFFFu) >= top || most >> 16 >= top) != 0;
      }
      if (!odd) {
        u32x4 vf[kRing];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) vf[n] = value_operand(n);
#pragma unroll
        for (int n = 0; n < NB * ND; ++n) {
          if (n + kAhead < NB * ND) vf[(n + kAhead) % kRing] = value_operand(n + kAhead);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) o[n % ND][rt] = mfma<DT>(vf[n % kRing], pf[n / ND][rt], o[n % ND][rt]);
          keep_order();
        }
      } else {
        // Such values count as zeros in the product, and are added to the rows that see them.
#pragma unroll
        for (int n = 0; n < NB * ND; ++n) {
          u32x4 v = value_operand(n);
          drop_nonfinite<DT>(v);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) o[n % ND][rt] = mfma<DT>(v, pf[n / ND][rt], o[n % ND][rt]);
        }
        for (int j = max(at, from); j < min(at + KT, to); ++j) {
          const T* row = vb + (int64_t)j * a.v_stride[0] + lg * 4;
#pragma unroll
          for (int dt = 0; dt < ND; ++dt) {
            if (dt * 16 >= a.head_dim) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = Elem<DT>::load(row[dt * 16 + i]), add = fabsf(v) < INFINITY ? 0.f : v;
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                const bool seen = begin[rt] != kNowhere && begin[rt] <= j && j <= row0 + rt * 16 + (lane & 15);
                o[dt][rt][i] += seen ? add : 0.f;
              }
            }
          }
        }
      }
    }
    half ^= 1;
  }

#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float sum = groups_sum(z[rt]), inv = 1.f / sum;
    if (begin[rt] == kNowhere) continue;
    const int i = row0 + rt * 16 + (lane & 15);
    T* out = static_cast<T*>(a.out) + i * a.out_stride[0] + head * a.out_stride[1] + lg * 4;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt)
      if (dt * 16 < a.head_dim) {
        const f32x4 v = sum == 0.f ? f32x4(0.f) : o[dt][rt] * inv;
        *reinterpret_cast<u32x2*>(out + dt * 16) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
      }
  }
}

namespace {

// Row tiles of a wave: two, but one at 256 columns, whose outputs fill the registers, and where workgroups of 128 tokens
// would be so few (three a CU, four at 64 columns) that the longest is waited for. One against two, us on the
// GPU: 8 prompts of 2048 tokens, 32 heads over 8 of 128, 4096 workgroups 364 / 300; 4 of 1000, 1024 workgroups 73 / 68
// (at 64 columns 2 of 2000 59 / 71); one of 2050, 544 workgroups 59 / 75; one of 300, 96 workgroups 11.7 / 14.7; one of 77
// 6.7 / 8.4.
int row_tiles_of(const tf_exl3_prompt_attention_args& a) {
  const int64_t two = ((int64_t)a.tokens + 32 * kPromptWaves - 1) / (32 * kPromptWaves) * a.q_heads;
  return a.head_dim > 128 || two <= (a.head_dim <= 64 ? 1024 : 768) ? 1 : 2;
}

int64_t tiles_of(const tf_exl3_prompt_attention_args& a) {
  const int rows = 16 * row_tiles_of(a) * kPromptWaves;
  return ((int64_t)a.tokens + rows - 1) / rows;
}

template <int DT, int DP, int RT, int KT>
void launch_rows(const tf_exl3_prompt_attention_args& a, const PromptPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((prompt_attention_kernel<DT, DP, RT, KT>), dim3((unsigned)(tiles_of(a) * a.q_heads)), dim3(kPromptThreads), 0,
                     stream, a, p);
}

template <int DT>
void launch(const tf_exl3_prompt_attention_args& a, const PromptPlan& p, hipStream_t stream) {
  const bool one = row_tiles_of(a) == 1;
  if (a.head_dim <= 64)
    one ? launch_rows<DT, 64, 1, 64>(a, p, stream) : launch_rows<DT, 64, 2, 64>(a, p, stream);
  else if (a.head_dim <= 128)
    one ? launch_rows<DT, 128, 1, 64>(a, p, stream) : launch_rows<DT, 128, 2, 64>(a, p, stream);
  else
    launch_rows<DT, 256, 1, 32>(a, p, stream);
}

}  // namespace

bool prompt_attention_fits(const tf_exl3_prompt_attention_args& a) { return launchable(tiles_of(a) * a.q_heads, kPromptThreads); }

hipError_t launch_prompt_attention(const tf_exl3_prompt_attention_args& a, hipStream_t stream) {
  PromptPlan p;
  p.tiles = (int)tiles_of(a);
  p.spread = a.q_heads % kXCDs == 0 ? a.q_heads / kXCDs : 0;
  p.by_heads = fast_div(p.spread ? p.spread : a.q_heads), p.by_group = fast_div(a.q_heads / a.kv_heads);
  // A scale of 0 keeps masked scores apart from others: the smallest factor does the same to sums.
  const float c = fabsf(a.scale) * 1.4426950408889634f;
  p.c = c > 1.2e-38f ? c : 1.2e-38f;
  const float slack = a.dtype == TF_DT_F16 ? Weights<TF_DT_F16>::kSlack : Weights<TF_DT_BF16>::kSlack;
  p.slack = fminf(slack / p.c, 3e38f);
  p.negate = a.scale < 0.f;
  if (a.dtype == TF_DT_F16)
    launch<TF_DT_F16>(a, p, stream);
  else
    launch<TF_DT_BF16>(a, p, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
