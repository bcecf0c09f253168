// Causal attention over packed prompts with grouped heads:
//
//   row r of sequence i (of ql rows) sees keys 0 .. r + kl - ql (of kl keys)
//   s_j = scale * q_r . k_j,   y_r = sum_j softmax(s)_j v_j
//
// A row that sees no key gives 0 (and -inf as its log-sum).
//
// The rows of a tile are (token, head of the group) pairs: the query heads
// that share a key-value head are stacked, token by token, so that each key
// tile is read once for the group and the causal border wastes little of a
// tile.  The scores of a tile never leave the SM: one pass over the keys with
// the running maximum and sum of each row.
#include "attention.cuh"

namespace bitnet {

struct AttnPromptArgs {
  const uint16_t* q;      // [Tq, Hq, D], tokens q_stride elements apart
  const uint16_t* k;      // [Tk, Hkv, D], tokens k_stride apart
  const uint16_t* v;
  const int32_t* cu_q;    // [B + 1] first row of each sequence
  const int32_t* cu_k;    // [B + 1] first key
  uint16_t* y;            // [Tq, Hq, D], tokens y_stride apart
  float* lse;             // [Tq, Hq] or null
  int64_t q_stride, k_stride, v_stride, y_stride;
  int B, Tq, Tk, Hq, Hkv, group;
  int tile_tokens;        // tokens per tile
  int half_tokens;        // tile kernel: tokens per 128 rows
  float scale, scale_log2;   // scale_log2 = scale * log2(e)
};

// One tile of work: rows [t0, t0 + n) of a sequence.
struct PromptTile {
  int q0, ql, k0, kl;     // the sequence
  int t0;                 // first token of the tile within it
  int ok;
};

// Tile number x, counted from the last tile of the last sequence backwards
// (late tiles see the most keys: the longest work starts first).  Called by a
// whole warp.  Sequences whose bounds are not inside the arrays have no tiles;
// `record` reports them.
__device__ __forceinline__ PromptTile prompt_find_tile(const AttnPromptArgs& a, int x,
                                                       bool record) {
  const int lane = threadIdx.x & 31;
  PromptTile t{};
  int seen = 0;
  for (int base = a.B - 1; base >= 0; base -= 32) {
    const int i = base - lane;
    int n = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    if (i >= 0) {
      q0 = a.cu_q[i]; q1 = a.cu_q[i + 1];
      k0 = a.cu_k[i]; k1 = a.cu_k[i + 1];
      if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) {
        if (record) record_error(BITNET_ERR_INVALID_ARG);
      } else {
        n = (q1 - q0 + a.tile_tokens - 1) / a.tile_tokens;
      }
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x < seen + inc);
    if (hit) {
      const int src = __ffs(hit) - 1;
      t.q0 = __shfl_sync(0xffffffffu, q0, src);
      t.ql = __shfl_sync(0xffffffffu, q1 - q0, src);
      t.k0 = __shfl_sync(0xffffffffu, k0, src);
      t.kl = __shfl_sync(0xffffffffu, k1 - k0, src);
      const int ns = __shfl_sync(0xffffffffu, n, src);
      const int first = seen + __shfl_sync(0xffffffffu, inc, src) - ns;
      const int at = x - first;              // outside [0, ns) only if bad bounds overflow the count
      t.t0 = (ns - 1 - at) * a.tile_tokens;
      t.ok = at >= 0 && at < ns;
      if (!record) return t;
      x = 0x7fffffff;                        // go on for the checks alone
    }
    seen += __shfl_sync(0xffffffffu, inc, 31);
  }
  return t;
}

// q . k of one row of D values each (16-byte aligned), in fp32.
template <int D>
__device__ __forceinline__ float row_dot(const uint16_t* q, const uint16_t* k) {
  float dot = 0.f;
#pragma unroll 8
  for (int d = 0; d < D; d += 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(q + d), y = *reinterpret_cast<const uint4*>(k + d);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dot += __uint_as_float(xs[i] << 16) * __uint_as_float(ys[i] << 16);
      dot += __uint_as_float(xs[i] & 0xffff0000u) * __uint_as_float(ys[i] & 0xffff0000u);
    }
  }
  return dot;
}

// Mends one row of y, by one warp, where the tiled result is not finite.  There
// are four ways to that besides values that the row sees.
//  * A masked probability (0) times an infinite or NaN value of the same sequence
//    gives NaN: such a value is then among the masked keys that the tile
//    multiplied, [seen, n_end), and no NaN among the seen ones.
//  * The sum of p v before the division passes fp32's range, with values near its
//    end: the column is then infinite without an infinity of that sign among the
//    seen values.  Columns of these two kinds are computed again, in fp32 with
//    the masked keys skipped and weights that are divided first; others stay.
//  * All scores are -inf (no_weight): the row is 0 whatever the values are.
//  * The row's sum is NaN (whole).  A score that is NaN or +inf gives that, and the
//    row stays NaN; and so do scores that the tile could not hold (see kPtFar),
//    whose row and log-sum are computed from the start.
// Lane i has columns i D / 32 onwards.
// 4096 tokens of 20 heads (92 us): a NaN or an infinity in a value that nearly all
// rows see 0.4 ms, all values NaN 0.6, a NaN key near the start or all queries NaN
// 0.4; in the middle, a NaN key 9.5 ms, an infinite value 16, a NaN value 11, and
// 35 at position 4000 (the rows just before it, few and long); a column of
// infinities 38, all scores far from 0 30.  Computing every such row as a whole
// took 77 .. 92 ms.
template <int D>
__device__ __noinline__ void prompt_row_by_warp(const AttnPromptArgs& a, const PromptTile& t,
                                                int token, int head, int n_end, bool no_weight,
                                                bool whole) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int kvh = head / a.group;
  const uint16_t* q = a.q + (int64_t)(t.q0 + token) * a.q_stride + (int64_t)head * D;
  const uint16_t* k = a.k + (int64_t)t.k0 * a.k_stride + (int64_t)kvh * D;
  const uint16_t* v = a.v + (int64_t)t.k0 * a.v_stride + (int64_t)kvh * D + lane * V;
  uint16_t* yr = a.y + (int64_t)(t.q0 + token) * a.y_stride + (int64_t)head * D + lane * V;
  const int seen = max(0, token + t.kl - t.ql + 1);
  auto columns = [](const uint16_t* p, uint32_t (&x)[V]) {   // this lane's of one row
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(p)[i / 2];
      x[i] = w & 0xffffu;
      x[i + 1] = w >> 16;
    }
  };
  if (no_weight) {
#pragma unroll
    for (int i = 0; i < V; i += 2) *reinterpret_cast<uint32_t*>(yr + i) = 0u;
    return;
  }
  uint32_t y[V], nans = 0, infs = 0, need = 0, found = 0;   // a bit per column
  columns(yr, y);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    nans |= (uint32_t)((y[i] & 0x7fffu) > 0x7f80u) << i;
    infs |= (uint32_t)((y[i] & 0x7fffu) == 0x7f80u) << i;
  }
  if (whole) {
    nans = infs = 0;
    found = ~0u;
  }
  if (__any_sync(0xffffffffu, nans != 0)) {
#pragma unroll 8
    for (int j = seen; j < n_end; ++j) {
      uint32_t x[V];
      columns(v + (int64_t)j * a.v_stride, x);
#pragma unroll
      for (int i = 0; i < V; ++i) need |= (uint32_t)((x[i] & 0x7f80u) == 0x7f80u) << i;
    }
    need &= nans;
  }
  need |= infs;
  // what the row sees may explain the column: an infinity of that sign, a NaN
  for (int j0 = 0; j0 < seen && __any_sync(0xffffffffu, (need & ~found) != 0); j0 += 32) {
#pragma unroll 8
    for (int j = j0; j < min(j0 + 32, seen); ++j) {
      uint32_t x[V];
      columns(v + (int64_t)j * a.v_stride, x);
#pragma unroll
      for (int i = 0; i < V; ++i)
        found |= (uint32_t)(infs >> i & 1u ? x[i] == y[i] : (x[i] & 0x7fffu) > 0x7f80u) << i;
    }
  }
  need = whole ? ~0u : need & ~found;
  if (!__any_sync(0xffffffffu, need != 0)) return;
  const float c = a.scale_log2;
  float m = -INFINITY, l = 0.f, o[V];
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const float s = j0 + lane < seen ? row_dot<D>(q, k + (int64_t)(j0 + lane) * a.k_stride) : -INFINITY;
    const float top = fmaxf(m, warp_max(s));
    if (__any_sync(0xffffffffu, !(s < INFINITY))) return;   // NaN, as it stands
    l = l * (m == top ? 1.f : ex2((m - top) * c)) + ex2((s - (top == -INFINITY ? 0.f : top)) * c);
    m = top;
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = 1.f / l;
  if (whole && a.lse && lane == 0)
    a.lse[(int64_t)(t.q0 + token) * a.Hq + head] = fmaf(m, a.scale, logf(l));
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 < seen; j0 += 32) {
    float p = 0.f;
    if (j0 + lane < seen)
      p = ex2((row_dot<D>(q, k + (int64_t)(j0 + lane) * a.k_stride) - m) * c) * inv;
    for (int x0 = 0; x0 < 32; x0 += 8) {     // eight rows of values on their way
      uint32_t w[8][V] = {};
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (j0 + x0 + x < seen) columns(v + (int64_t)(j0 + x0 + x) * a.v_stride, w[x]);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float px = __shfl_sync(0xffffffffu, p, x0 + x);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] += px * __uint_as_float(w[x][i] << 16);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (need >> i & 1u) yr[i] = (uint16_t)pack_bf16(o[i], 0.f);
}

constexpr int kPwRows = 64, kPwKeys = 64;    // rows and keys per tile
template <int D>
constexpr int pw_smem_bytes() { return (kPwRows + 4 * kPwKeys) * D * 2; }

// 4 warps of 16 rows each, mma.sync, keys and values double buffered by
// asynchronous copies.
template <int D>
__global__ void __launch_bounds__(128, 2) prompt_warp_kernel(const AttnPromptArgs a) {
  extern __shared__ __align__(128) uint8_t psm[];
  __shared__ PromptTile s_tile;
  constexpr int CH = D / 8, KT = D / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, mi = lane >> 3;
  pdl_wait();
  pdl_launch_dependents();
  const int kvh = blockIdx.x % a.Hkv;
  if (warp == 0) {
    const PromptTile f = prompt_find_tile(a, blockIdx.x / a.Hkv, blockIdx.x == 0);
    if (lane == 0) s_tile = f;
  }
  __syncthreads();
  const PromptTile t = s_tile;
  if (!t.ok) return;
  const int tokens = min(a.tile_tokens, t.ql - t.t0);
  const int rows = tokens * a.group;
  const int shift = t.kl - t.ql;             // row r sees keys 0 .. r + shift
  const int n_keys = max(0, min(t.kl, t.t0 + tokens + shift));   // seen by the last row
  const int n_tiles = (n_keys + kPwKeys - 1) / kPwKeys;
  const uint32_t qs = smem_u32(psm), ks = qs + kPwRows * D * 2, vs = ks + 2 * kPwKeys * D * 2;

  for (int x = tid; x < kPwRows * CH; x += 128) {
    const int r = x / CH, c = x % CH;
    const bool ok = r < rows;
    const int token = ok ? r / a.group : 0;
    const uint16_t* src = a.q + (int64_t)(t.q0 + t.t0 + token) * a.q_stride +
                          (int64_t)(kvh * a.group + (ok ? r % a.group : 0)) * D + c * 8;
    cp_async16(tile_addr<D>(qs, r, c), src, ok ? 16u : 0u);
  }
  auto load = [&](int j) {
    if (j < n_tiles) {
      const uint32_t kd = ks + (uint32_t)((j & 1) * kPwKeys * D * 2);
      const uint32_t vd = vs + (uint32_t)((j & 1) * kPwKeys * D * 2);
      for (int x = tid; x < kPwKeys * CH; x += 128) {
        const int r = x / CH, c = x % CH, key = j * kPwKeys + r;
        const bool ok = key < n_keys;
        const int64_t row = t.k0 + (ok ? key : 0);
        cp_async16(tile_addr<D>(kd, r, c), a.k + row * a.k_stride + (int64_t)kvh * D + c * 8,
                   ok ? 16u : 0u);
        cp_async16(tile_addr<D>(vd, r, c), a.v + row * a.v_stride + (int64_t)kvh * D + c * 8,
                   ok ? 16u : 0u);
      }
    }
    cp_async_commit();
  };
  load(0);

  float o[2 * KT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2 * KT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  uint32_t qf[KT][4];
  const int r0 = warp * 16 + (lane >> 2);    // this lane's rows: r0 and r0 + 8
  // last key each row sees
  const int lim0 = t.t0 + r0 / a.group + shift, lim1 = t.t0 + (r0 + 8) / a.group + shift;
  for (int j = 0; j < n_tiles; ++j) {
    load(j + 1);
    cp_async_wait<1>();
    __syncthreads();
    if (j == 0) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        ldsm_x4(tile_addr<D>(qs, warp * 16 + (lane & 7) + (mi & 1) * 8, kt * 2 + (mi >> 1)),
                qf[kt]);
    }
    const uint32_t kd = ks + (uint32_t)((j & 1) * kPwKeys * D * 2);
    const uint32_t vd = vs + (uint32_t)((j & 1) * kPwKeys * D * 2);
    float s[kPwKeys / 8][4];
#pragma unroll
    for (int nt = 0; nt < kPwKeys / 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int nt = 0; nt < kPwKeys / 8; nt += 2) {
        uint32_t bf[4];                      // keys nt*8 .. +15, two 8-wide steps of D
        ldsm_x4(tile_addr<D>(kd, nt * 8 + (lane & 7) + (mi >> 1) * 8, kt * 2 + (mi & 1)), bf);
        mma_bf16(s[nt], qf[kt], bf[0], bf[1]);
        mma_bf16(s[nt + 1], qf[kt], bf[2], bf[3]);
      }
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < kPwKeys / 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = j * kPwKeys + nt * 8 + 2 * (lane & 3) + (e & 1);
        s[nt][e] = key <= (e < 2 ? lim0 : lim1) && key < n_keys ? s[nt][e] : -INFINITY;
        if (e < 2) t0 = fmaxf(t0, s[nt][e]); else t1 = fmaxf(t1, s[nt][e]);
      }
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
    }
    t0 = fmaxf(t0, m[0]);
    t1 = fmaxf(t1, m[1]);
    const float c = a.scale_log2;
    const float f0 = m[0] == t0 ? 1.f : ex2((m[0] - t0) * c), f1 = m[1] == t1 ? 1.f : ex2((m[1] - t1) * c);
    m[0] = t0;
    m[1] = t1;
    l[0] *= f0;
    l[1] *= f1;
#pragma unroll
    for (int i = 0; i < 2 * KT; ++i) {
      o[i][0] *= f0;
      o[i][1] *= f0;
      o[i][2] *= f1;
      o[i][3] *= f1;
    }
    const float z0 = t0 == -INFINITY ? 0.f : t0, z1 = t1 == -INFINITY ? 0.f : t1;
#pragma unroll
    for (int nt = 0; nt < kPwKeys / 8; ++nt) {
      s[nt][0] = ex2((s[nt][0] - z0) * c);
      s[nt][1] = ex2((s[nt][1] - z0) * c);
      s[nt][2] = ex2((s[nt][2] - z1) * c);
      s[nt][3] = ex2((s[nt][3] - z1) * c);
      l[0] += s[nt][0] + s[nt][1];
      l[1] += s[nt][2] + s[nt][3];
    }
#pragma unroll
    for (int kk = 0; kk < kPwKeys / 16; ++kk) {
      uint32_t pf[4] = {pack_bf16(s[2 * kk][0], s[2 * kk][1]), pack_bf16(s[2 * kk][2], s[2 * kk][3]),
                        pack_bf16(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                        pack_bf16(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        uint32_t bf[4];                      // dims kt*16 .. +15 of keys kk*16 .. +15
        ldsm_x4_trans(tile_addr<D>(vd, kk * 16 + (lane & 7) + (mi & 1) * 8, kt * 2 + (mi >> 1)), bf);
        mma_bf16(o[2 * kt], pf, bf[0], bf[1]);
        mma_bf16(o[2 * kt + 1], pf, bf[2], bf[3]);
      }
    }
    __syncthreads();                         // the buffers may be refilled
  }
  cp_async_wait<0>();
  unsigned redo = 0, none = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    const int r = r0 + 8 * half;
    const float inv = l[half] == 0.f ? 0.f : 1.f / l[half];
    float odd = 0.f;
    if (r < rows) {
      const int64_t token = t.q0 + t.t0 + r / a.group;
      const int head = kvh * a.group + r % a.group;
      uint16_t* yr = a.y + token * a.y_stride + (int64_t)head * D;
#pragma unroll
      for (int i = 0; i < 2 * KT; ++i) {
        const float x0 = o[i][2 * half] * inv, x1 = o[i][2 * half + 1] * inv;
        odd += x0 * 0.f + x1 * 0.f;
        *reinterpret_cast<uint32_t*>(yr + i * 8 + 2 * (lane & 3)) = pack_bf16(x0, x1);
      }
      if (a.lse && (lane & 3) == 0)
        a.lse[token * a.Hq + head] =
            l[half] == 0.f ? -INFINITY : fmaf(m[half], a.scale, logf(l[half]));
    }
    // a sum that is NaN makes the whole row NaN, which it is already
    unsigned nan = __ballot_sync(0xffffffffu, odd != odd && l[half] == l[half]);
    nan |= nan >> 1;
    nan |= nan >> 2;
    redo = (nan & 0x11111111u) << half | redo;   // bit 4 i + half: row i + 8 half of the warp
    none |= (__ballot_sync(0xffffffffu, l[half] == 0.f) & 0x11111111u) << half;
  }
  while (redo) {
    const int bit = __ffs(redo) - 1;
    redo &= redo - 1;
    const int r = warp * 16 + (bit >> 2) + 8 * (bit & 3);
    __syncwarp();
    prompt_row_by_warp<D>(a, t, t.t0 + r / a.group, kvh * a.group + r % a.group, n_keys,
                          none >> bit & 1u, false);
  }
}


// ------------------------------------------------------------ tensor cores
//
// The tile kernel: 2 x 128 rows per CTA on tcgen05.  Twenty warps:
//   * 16 softmax warps, 8 for each 128 rows: a thread has one row (a TMEM
//     lane) and half of a step's columns, so four of them share a scheduler
//     and hide each other's latencies;
//   * warp 16 (one thread): TMA loads of Q once and of K, V tiles of 128 keys
//     into a ring;
//   * warp 17 (one thread): the MMAs.
// Per step of 64 keys and row half i:
//   S_i = Q_i K^T    both operands in shared memory, fp32 scores in one of two
//                    buffers in TMEM
//   P_i = exp2(c S_i - m_i)   read by the softmax threads, written back over
//                    the scores as bf16 pairs (32 of their 64 columns)
//   O_i += P_i V     P_i from TMEM, V (rows of D values, so MN-major) from
//                    shared memory, fp32 sums in TMEM
// The scores of a half are two steps ahead of its outputs, so the softmax
// warps find the next scores when they have done with the last.  MMAs are
// executed in issue order: the scores of step u + 2 may overwrite P of step u
// as soon as they are issued after its product.
//
// The reference m_i of a row only has to keep the exponentials in range, not
// to be the running maximum: the result is divided by the same scaled sum.  So
// a step's exponentials are taken with the reference of the steps before it
// while its own maximum is still being found, and only if a row outgrows its
// reference by 2^8 (always in the first step) is the step done again, with
// O_i rescaled.  bf16 has fp32's range, so probabilities up to 2^8 lose
// nothing.
//
// Measured (device time, the same inputs again and again): 4096 tokens of 20
// heads of 128 on 4 key-value heads 90 us (955 TFLOP/s; 103 on inputs that
// change from call to call), 16384 tokens 1.14 ms, 1.31 under the power cap
// (1200, 1050), 4096 tokens of 16 heads of 64 61 us.  Every CTA searches its
// tile in the bounds, 32 sequences at a time, which shows with hundreds of
// them: 200 prompts of 32 tokens 75 us, 1000 of them 709.  A step of both
// halves takes about 1850 cycles with D = 128.  Its MMAs back to back take 1239
// (the score MMAs read Q and K from shared memory at its full 128 bytes a
// clock, so 48 cycles instead of 32 for 128 x 64 x 16); with the barriers
// handed over but no softmax 1560; taking the ring's TMA traffic away changes
// nothing.  The four softmax warps of a scheduler need 1024 cycles for the
// exponentials alone (4 a clock), which is the bound with D = 64.  What the
// issuing thread does between MMAs counts: its loop is unrolled over halves and
// steps, one thread issues everything.
// Alternatives, 4096 tokens of 20 heads: scores 128 keys wide and single
// buffered (a half's softmax and MMAs in turn) 97 us; one thread per whole row
// (8 softmax warps) 105 us and more; two issuing warps, one per half (the
// halves fall into step and wait for the same unit) 108 us; a quarter of the
// exponentials as polynomials on the fp32 pipe 104 us (against 99 then); waits
// that poll in a plain loop 101 us.
constexpr int kPtKeys = 128, kPtSub = 64;
constexpr int kPtThreads = 640;
constexpr int kPtRegs = 96;                  // 65536 / 640, in steps of 8
// The exponents are fma(s, c, -(c m)) with c m rounded before.  That rounding
// is the same for the whole row and leaves its result while it is small against
// fp32's range of exponents: at most 32 below |c m| = 2^30.  Rows whose
// reference was ever farther from 0 get NaN as their sum and are computed again
// by prompt_row_by_warp, which subtracts first.  Doing that here costs every step
// of every row: 4096 tokens of 20 heads 92 -> 98 us with the subtraction, 95 with
// a second loop for such rows, 94 with a factor c per row that makes the product
// exact.
constexpr float kPtFar = 1073741824.0f;
template <int D>
struct PtCfg {
  static constexpr int kHalves = D / 64;                  // 128-byte wide column blocks
  static constexpr int kBlock = 128 * 128;                // 128 rows of 64 bf16
  static constexpr int kTile = kHalves * kBlock;          // a Q half, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kBars = 2 * kStages + 14;
  static constexpr int kExch = 2 * 2 * 128 * 4;           // a float per softmax thread
  static constexpr size_t kSmem = (size_t)(2 + kStages) * kTile + kExch + kBars * 8 + 64;
  // D fp32, A and B bf16, M 128; scores: N 64, both K-major; outputs: N = D, B MN-major
  static constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) |
                                      ((uint32_t)(kPtSub >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                      ((uint32_t)(D >> 3) << 17) | (8u << 24);
};

// Barrier of the two warps that share 32 rows; `any` tells whether the
// condition holds in one of their threads.
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool pair_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

// Shared-memory descriptor of an MN-major operand in 128-byte swizzled rows:
// 64 columns per 128-byte row, the next 64 columns `block` bytes on, 8 rows
// (of the contraction) per 1024 bytes.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3fffu);
  d |= (uint64_t)(block >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
__device__ __forceinline__ void tc_mma_bf16(uint32_t dtmem, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t dtmem, uint32_t a_tmem, uint64_t bdesc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(dtmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// 32 columns of this warp's 32 lanes; the registers are valid after
// tcgen05.wait::ld.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32_async(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15])
      : "memory");
}
// Waits for this thread's loads; the 32 registers pass through it, so no use
// of them can be scheduled before the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Two fp32 lanes in one 64-bit register pair.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// True in one lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}
// The largest of three, NaN if one of them is NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int D>
__global__ void __launch_bounds__(kPtThreads, 1)
    prompt_tile_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const AttnPromptArgs a) {
  using C = PtCfg<D>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];      // the swizzled tiles come first
  uint8_t* ring = smem + 2 * C::kTile;
  float* exch = reinterpret_cast<float*>(ring + (size_t)S * C::kTile);   // [2 halves][2][128]
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(exch + C::kExch / 4);
  uint64_t* kv_empty = kv_full + S;
  uint64_t* q_full = kv_empty + S;
  uint64_t* s_full = q_full + 1;             // [2 halves][2 buffers]
  uint64_t* p_full = s_full + 4;             // [2][2]
  uint64_t* o_done = p_full + 4;             // [2] after every step
  uint64_t* o_full = o_done + 2;             // [2] after the last one
  uint64_t* v_clean = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_full + C::kBars);
  PromptTile* s_tile = reinterpret_cast<PromptTile*>(tmem_slot + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int kvh = blockIdx.x % a.Hkv;
  if (tid == 512) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(v_clean, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&o_done[i], 1);
      mbar_init(&o_full[i], 1);
    }
    fence_mbar_init();
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (smem_u32(smem) & 1023u) {              // the swizzle counts on it
    if (tid == 0) record_error(BITNET_ERR_UNSUPPORTED);
    return;
  }
  if (warp == 0) {
    pdl_wait();
    const PromptTile f = prompt_find_tile(a, blockIdx.x / a.Hkv, blockIdx.x == 0);
    if (lane == 0) *s_tile = f;
  } else if (warp == 17) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const PromptTile t = *s_tile;
  if (tid == 0) pdl_launch_dependents();
  if (!t.ok) {
    if (warp == 17)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                   : "memory");
    return;
  }

  // the two halves: tokens and steps of 64 keys
  const int half_tokens = a.half_tokens;
  const int end = min(t.t0 + a.tile_tokens, t.ql);         // the tile may be one half long
  const int shift = t.kl - t.ql;             // row r sees keys 0 .. r + shift
  int n_steps[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int first = t.t0 + i * half_tokens;
    const int last = min(first + half_tokens, end) - 1;
    const int keys = last < first ? 0 : max(0, min(t.kl, last + shift + 1));
    n_steps[i] = (keys + kPtSub - 1) / kPtSub;
  }
  const int n_all = max(n_steps[0], n_steps[1]);
  // the last tile of values reaches behind the sequence
  const int last_tile = (n_all - 1) >> 1;
  const bool v_tail = n_all > 0 && (last_tile + 1) * kPtKeys > t.kl;

  if (warp >= 16) {
    if (warp == 16 && n_all > 0) {
      // ------------------------------------------------------ TMA producer
      bool ok = true;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(2 * C::kHalves * half_tokens * a.group * 128));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(smem_u32(smem) + (uint32_t)(i * C::kTile + h * C::kBlock), &tq, q_full,
                        h * 64, kvh * a.group, t.q0 + t.t0 + i * half_tokens);
        int u = 0;                           // tiles K_0 V_0 K_1 V_1 ...
        for (; u < 2 * (last_tile + 1); ++u) {
          const int s = u % S;
          if (u >= S && !mbar_wait(&kv_empty[s], ((u / S) - 1) & 1)) { ok = false; break; }
          mbar_arrive_expect_tx(&kv_full[s], (uint32_t)C::kTile);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(smem_u32(ring) + (uint32_t)(s * C::kTile + h * C::kBlock),
                        (u & 1) ? &tv : &tk, &kv_full[s], h * 64, kvh, t.k0 + (u >> 1) * kPtKeys);
        }
        // a wait that gave up: the copies in flight still land before the exit
        if (!ok)
          for (int w = u > S ? u - S : 0; w < u; ++w) mbar_wait(&kv_full[w % S], (w / S) & 1);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (ok && v_tail) {
        // values behind the sequence (another's, or whatever lies there) are
        // zeroed, so that a masked probability times one of them is 0
        const int e = 2 * last_tile + 1, r0 = t.kl - last_tile * kPtKeys;
        if (__all_sync(0xffffffffu, mbar_wait(&kv_full[e % S], (uint32_t)((e / S) & 1)))) {
          for (int x = r0 * 8 + lane; x < kPtKeys * 8; x += 32)        // rows of 128 bytes
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              sts_v4(smem_u32(ring) + (uint32_t)((e % S) * C::kTile + h * C::kBlock + x * 16),
                     make_uint4(0u, 0u, 0u, 0u));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_clean);
        }
      }
    } else if (warp == 17 && elect_one() && n_all > 0) {
      // -------------------------------------------------------- MMA issuer
      const uint64_t q_desc = sw128_desc(smem_u32(smem)), k_desc = sw128_desc(smem_u32(ring));
      const uint64_t v_desc = sw128_mn_desc(smem_u32(ring), C::kBlock);
      // S_i[b] = Q_i K^T, the 64 keys of step b of the tile at k_tile
      auto scores = [&](int i, int b, uint64_t k_tile) {
        const uint64_t qd = q_desc + (uint64_t)(i * (C::kTile >> 4));
        const uint64_t kd = k_tile + (uint64_t)(b * (kPtSub * 128 >> 4));
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint64_t o = (uint64_t)((x >> 2) * (C::kBlock >> 4) + 2 * (x & 3));
          tc_mma_bf16(tmem + (uint32_t)(i * 128 + b * kPtSub), qd + o, kd + o, C::kIdescS, x > 0);
        }
        tc_commit(&s_full[2 * i + b]);
      };
      // O_i (+)= P_i[b] V, the 64 values of step b of the tile at v_tile
      auto outputs = [&](int i, int b, uint64_t v_tile, bool add) {
        const uint64_t vd = v_tile + (uint64_t)(b * (kPtSub * 128 >> 4));
        const uint32_t ot = tmem + (uint32_t)(256 + i * D);
        const uint32_t pt = tmem + (uint32_t)(i * 128 + b * kPtSub);
        tc_mma_bf16_ts(ot, pt, vd, C::kIdescO, add);
#pragma unroll
        for (int x = 1; x < kPtSub / 16; ++x)
          tc_mma_bf16_ts(ot, pt + 8 * x, vd + x * (2048 >> 4), C::kIdescO, 1);
        tc_commit(&o_done[i]);
      };
      // scores run two steps ahead of the outputs; K of tile j and V of tile j
      // are ring entries 2 j and 2 j + 1
      const int n0 = n_steps[0], n1 = n_steps[1];
      bool ok = mbar_wait(q_full, 0) && mbar_wait(&kv_full[0], 0);
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (b < (i ? n1 : n0)) scores(i, b, k_desc);
        tc_commit(&kv_empty[0]);
      }
      int s = 1;                             // stage and phase of V_j
      uint32_t ph = 0;
      for (int j = 0; j <= last_tile && ok; ++j) {
        const int sk = s + 1 == S ? 0 : s + 1;               // K_{j+1}
        const uint32_t phk = s + 1 == S ? ph ^ 1 : ph, par = (uint32_t)(j & 1);
        const uint64_t v_tile = v_desc + (uint64_t)(s * (C::kTile >> 4));
        const uint64_t k_tile = k_desc + (uint64_t)(sk * (C::kTile >> 4));
        ok = mbar_wait(&kv_full[s], ph) && (j == last_tile || mbar_wait(&kv_full[sk], phk)) &&
             (!v_tail || j < last_tile || mbar_wait(v_clean, 0));
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int left = (i ? n1 : n0) - 2 * j - b;      // steps from this one on
            if (!ok || left <= 0) continue;
            ok = mbar_wait(&p_full[2 * i + b], par);
            if (!ok) continue;
            tc_fence_after();
            outputs(i, b, v_tile, j + b > 0);
            if (left > 2) scores(i, b, k_tile);
            if (left == 1) tc_commit(&o_full[i]);
          }
        if (ok) {
          tc_commit(&kv_empty[s]);
          if (j < last_tile) tc_commit(&kv_empty[sk]);
        }
        s = sk + 1 == S ? 0 : sk + 1;
        ph = sk + 1 == S ? phk ^ 1 : phk;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    // The registers the launch gave (no more are asked for; the host checks that
    // the build has them).  Without the statement the compiler schedules the loop
    // below worse: 4096 tokens of 20 heads 91.8 instead of 87.9 us.  Giving the
    // softmax warps 104 and the others 64 spills in the issuing thread: 98 us.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPtRegs));
    const int i = warp >> 3, cg = (warp >> 2) & 1;       // row half, column half
    const int r = 32 * (warp & 3) + lane;    // this thread's row
    const int pair = 1 + 4 * i + (warp & 3);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t st = tmem + lanes + (uint32_t)(i * 128 + cg * 32);
    const uint32_t pt = tmem + lanes + (uint32_t)(i * 128 + cg * 16);
    const uint32_t ot = tmem + lanes + (uint32_t)(256 + i * D + cg * (D / 2));
    float* mine = exch + (2 * i + cg) * 128 + r;
    const float* other = exch + (2 * i + (cg ^ 1)) * 128 + r;
    const int n = i ? n_steps[1] : n_steps[0];
    const int first = t.t0 + i * half_tokens;
    const int token = first + r / a.group;
    const int lim = token + shift - cg * 32; // last key the row sees, from this column half
    const float c = a.scale_log2;
    const uint64_t c2 = f2_pack(c, c);
    const float slack = 8.0f / c;
    float m = -INFINITY;
    uint64_t l2[2] = {0, 0};                 // partial sums, two lanes each
    // a wait that gave up does not end the loop: both warps of a pair go on to
    // the same barriers (without further waits) and nothing is written
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int buf = 2 * i + (j & 1);
      const uint32_t sub = (uint32_t)((j & 1) * kPtSub);
      if (ok) ok = mbar_wait(&s_full[buf], (uint32_t)((j >> 1) & 1));
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const bool border = j * kPtSub + kPtSub - 1 > first + shift;   // some row ends inside
      const int e = lim - j * kPtSub;
      while (true) {
        const float neg = m == -INFINITY ? 0.0f : -m * c;
        const uint64_t neg2 = f2_pack(neg, neg);
        uint32_t s[32], p[16];
        float mx[2] = {-INFINITY, -INFINITY};
        uint64_t t2[2] = {0, 0};
        tmem_ld32_async(st + sub, s);
        tmem_wait_ld(s);
        if (border) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x > e) s[x] = 0xff800000u;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float s0 = __uint_as_float(s[2 * x]), s1 = __uint_as_float(s[2 * x + 1]);
          mx[x & 1] = max3_nan(mx[x & 1], s0, s1);
          const uint64_t y = f2_fma(f2_pack(s0, s1), c2, neg2);
          float e0, e1;
          f2_unpack(y, e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          p[x] = pack_bf16(e0, e1);
          t2[x & 1] = f2_add(t2[x & 1], f2_pack(e0, e1));
        }
        const float top = max3_nan(mx[0], mx[1], mx[1]);
        // the vote also says that both warps have read their scores, which P
        // is about to overwrite
        if (pair_any(pair, top > m + slack)) {
          // a row has outgrown its reference (or had none): once more with it
          *mine = top;
          pair_sync(pair);
          const float both = fmaxf(top, *other);
          const float to = both > m + slack ? both : m;
          const float f = to == m ? 1.0f : ex2((m - to) * c);
          m = to;
          if (j > 0) {
            // O holds the steps before this one once their MMAs are done
            // (these scores came after those of step j - 2, so the wait can
            // only be for step j - 1 and its parity is enough)
            if (ok) ok = mbar_wait(&o_done[i], (uint32_t)((j - 1) & 1));
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const uint64_t f2 = f2_pack(f, f);
            l2[0] = f2_fma(l2[0], f2, 0);
            l2[1] = f2_fma(l2[1], f2, 0);
#pragma unroll
            for (int x = 0; x < D / 2; x += 32) {
              uint32_t o[32];
              tmem_ld32_async(ot + x, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st32_async(ot + x, o);
            }
          }
          if (fabsf(m) < INFINITY && !(fabsf(m * c) < kPtFar)) l2[0] = f2_pack(NAN, NAN);
          continue;
        }
        tmem_st16_async(pt + sub, p);
        l2[0] = f2_add(l2[0], t2[0]);
        l2[1] = f2_add(l2[1], t2[1]);
        break;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[buf]);
    }
    // ------------------------------------------------------------ epilogue
    float l, l1;
    f2_unpack(f2_add(l2[0], l2[1]), l, l1);
    l += l1;
    *mine = l;
    pair_sync(pair);
    l += *other;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (n > 0)
      ok = ok && mbar_wait(&o_full[i], 0);
    else if (n_all > 0)
      ok = mbar_wait(q_full, 0);             // the copy into what becomes the staging area
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    // through shared memory (the half's Q tile, which every MMA has read) so
    // that whole segments of D / 2 values are written at a time; 16-byte chunks
    // are xored with the row
    constexpr int CH = D / 16;               // chunks per segment
    const int rows = (min(first + half_tokens, end) - first) * a.group;   // may be <= 0
    const uint32_t stage = smem_u32(smem) + (uint32_t)(i * C::kTile + (warp & 7) * 32 * D);
    auto at = [&](int row, int ch) {
      return stage + (uint32_t)(row * D + ((ch ^ ((row * CH / 8) & (CH - 1))) << 4));
    };
    float odd = 0.0f;
#pragma unroll
    for (int x = 0; x < D / 2; x += 32) {
      uint32_t o[32];
      if (n > 0) {
        tmem_ld32_async(ot + x, o);
        tmem_wait_ld(o);
      } else {
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = 0;
      }
#pragma unroll
      for (int y = 0; y < 32; y += 8) {
        float f[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          f[z] = __uint_as_float(o[y + z]) * inv;
          odd = fmaf(f[z], 0.0f, odd);
        }
        sts_v4(at(lane, (x + y) / 8), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                 pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
      }
    }
    __syncwarp();
    const int r0 = 32 * (warp & 3);
    if (ok) {
      const uint32_t inv_group = (65536u + (uint32_t)a.group - 1) / (uint32_t)a.group;
#pragma unroll
      for (int y = 0; y < CH; ++y) {
        const int x = y * 32 + lane, rr = x / CH, ch = x % CH, row = r0 + rr;
        if (row < rows) {
          // row / group, exact for rows below 128 and groups up to 64
          const int tok = (int)(((uint32_t)row * inv_group) >> 16);
          const int head = kvh * a.group + row - tok * a.group;
          *reinterpret_cast<uint4*>(a.y + (int64_t)(t.q0 + first + tok) * a.y_stride +
                                    (int64_t)head * D + cg * (D / 2) + ch * 8) = lds_v4(at(rr, ch));
        }
      }
      if (a.lse && cg == 0 && r < rows)
        a.lse[(int64_t)(t.q0 + token) * a.Hq + kvh * a.group + r % a.group] =
            l == 0.0f ? -INFINITY
                      : ((m == -INFINITY ? 0.0f : m * c) + log2f(l)) * 0.69314718055994531f;
    }
    // rows with a result that is not finite are looked at again, the pair's warps
    // taking turns; both warps' stores come first
    const bool mend = ok && r < rows && odd != odd;
    if (pair_any(pair, mend)) {
      *mine = mend ? 1.0f : 0.0f;
      pair_sync(pair);
      unsigned redo = __ballot_sync(0xffffffffu, *mine + *other > 0.0f);
      const unsigned none = __ballot_sync(0xffffffffu, l == 0.0f);
      const unsigned whole = __ballot_sync(0xffffffffu, l != l);
      for (int k = 0; redo; ++k) {
        const int bit = __ffs(redo) - 1, row = r0 + bit;
        redo &= redo - 1;
        if ((k & 1) == cg)
          prompt_row_by_warp<D>(a, t, first + row / a.group, kvh * a.group + row % a.group,
                                min(n * kPtSub, t.kl), none >> bit & 1u, whole >> bit & 1u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

}  // namespace bitnet
