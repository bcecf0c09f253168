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
  float scale_log2;       // scale * log2(e)
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
      t.t0 = (ns - 1 - (x - first)) * a.tile_tokens;
      t.ok = 1;
      if (!record) return t;
      x = 0x7fffffff;                        // go on for the checks alone
    }
    seen += __shfl_sync(0xffffffffu, inc, 31);
  }
  return t;
}

// One row by one warp in fp32 with the masked keys skipped: 32 keys at a time,
// one per lane for the scores, then one output column set per lane.  For rows
// whose tiled result is not finite: there a masked probability (0) times a
// value that is infinite or NaN gives NaN, and this gives the row's own value.
template <int D>
__device__ __noinline__ void prompt_row_by_warp(const AttnPromptArgs& a, const PromptTile& t,
                                                int token, int head) {
  const int lane = threadIdx.x & 31;
  const int kvh = head / a.group;
  const uint16_t* q = a.q + (int64_t)(t.q0 + token) * a.q_stride + (int64_t)head * D;
  const uint16_t* k = a.k + (int64_t)t.k0 * a.k_stride + (int64_t)kvh * D;
  const uint16_t* v = a.v + (int64_t)t.k0 * a.v_stride + (int64_t)kvh * D;
  const int n = token + t.kl - t.ql + 1;
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < n) {
      const uint16_t* kr = k + (int64_t)j * a.k_stride;
      float dot = 0.f;
      for (int d = 0; d < D; ++d) dot += bf16_bits_to_float(q[d]) * bf16_bits_to_float(kr[d]);
      s = dot * a.scale_log2;
    }
    const float top = fmaxf(m, warp_max(s));
    const float f = m == top ? 1.f : ex2(m - top);
    const float p = ex2(s - (top == -INFINITY ? 0.f : top));
    m = top;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f;
    for (int x = 0; x < 32 && j0 + x < n; ++x) {
      const float px = __shfl_sync(0xffffffffu, p, x);
      const uint16_t* vr = v + (int64_t)(j0 + x) * a.v_stride + lane * (D / 32);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] += px * bf16_bits_to_float(vr[i]);
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* yr = a.y + (int64_t)(t.q0 + token) * a.y_stride + (int64_t)head * D + lane * (D / 32);
#pragma unroll
  for (int i = 0; i < D / 32; i += 2)
    *reinterpret_cast<uint32_t*>(yr + i) = pack_bf16(o[i] * inv, o[i + 1] * inv);
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
        s[nt][e] = key <= (e < 2 ? lim0 : lim1) && key < n_keys ? s[nt][e] * a.scale_log2 : -INFINITY;
        if (e < 2) t0 = fmaxf(t0, s[nt][e]); else t1 = fmaxf(t1, s[nt][e]);
      }
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
    }
    t0 = fmaxf(t0, m[0]);
    t1 = fmaxf(t1, m[1]);
    const float f0 = m[0] == t0 ? 1.f : ex2(m[0] - t0), f1 = m[1] == t1 ? 1.f : ex2(m[1] - t1);
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
      s[nt][0] = ex2(s[nt][0] - z0);
      s[nt][1] = ex2(s[nt][1] - z0);
      s[nt][2] = ex2(s[nt][2] - z1);
      s[nt][3] = ex2(s[nt][3] - z1);
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
  unsigned redo = 0;
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
        a.lse[token * a.Hq + head] = l[half] == 0.f
                                         ? -INFINITY
                                         : (m[half] + log2f(l[half])) * 0.69314718055994531f;
    }
    unsigned nan = __ballot_sync(0xffffffffu, odd != odd);
    nan |= nan >> 1;
    nan |= nan >> 2;
    redo = (nan & 0x11111111u) << half | redo;   // bit 4 i + half: row i + 8 half of the warp
  }
  while (redo) {
    const int bit = __ffs(redo) - 1;
    redo &= redo - 1;
    const int r = warp * 16 + (bit >> 2) + 8 * (bit & 3);
    __syncwarp();
    prompt_row_by_warp<D>(a, t, t.t0 + r / a.group, kvh * a.group + r % a.group);
  }
}

}  // namespace bitnet
