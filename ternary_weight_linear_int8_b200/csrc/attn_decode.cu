// Attention of one new token per sequence over a paged key-value cache:
//
//   s_j = scale * q . k_j   over the lens[b] keys of the sequence
//   y   = sum_j p_j v_j,    p_j = exp(s_j - m) / sum_i exp(s_i - m)
//
// with Hq / Hkv query heads sharing each key-value head.  Every key and value
// is read once for all the query heads of its group, so the work is bound by
// the cache's bytes: 4 D Hkv per token.
//
// The caches of all sequences are cut into units of 64 tokens of one
// key-value head, numbered sequence by sequence and head by head, and every
// CTA takes an equal contiguous run of units, whatever the lengths are (they
// are known on the device only).  A run covers one or more (sequence, head)
// pairs, at most its first and last ones in part: whole ones are finished
// here, partial ones leave their maximum, sum and unnormalised output in the
// workspace and a second kernel joins them in a fixed order, so the result
// does not depend on timing.
//
// Inside a CTA each of 4 warps takes 16 tokens of every unit with its own
// ring of asynchronous copies (no block barrier between units) and its own
// running maximum, sum and output:
//   S^T [16 tokens x 8 heads] = K Q^T         mma.sync, K by ldmatrix
//   O^T [D x 8 heads]        += V^T P^T       V by ldmatrix.trans
// Keys are the M side because groups have at most 8 heads as a rule, so that
// the heads fill the 8-wide N side; P^T is S^T's accumulator transposed in
// registers (movmatrix).  P is rounded to bf16 for the second product (2^-8
// relative at most, like the outputs' own rounding); maxima, sums and
// outputs stay in fp32.
#include "attention.cuh"

namespace bitnet {

constexpr int kDecWarps = 4;
constexpr int kDecUnit = 16 * kDecWarps;   // tokens per unit
// CTAs per SM and stages of a warp's ring.  With D = 128 two CTAs of three
// stages of 8 KB (128 KB of copies ahead of the computation per SM); three of
// two stages are slower on long contexts (100003 tokens of 64 heads 71.9 -> 73.6
// us).  With D = 64 the same bytes are twice the tokens, and a third CTA hides
// more of each step's latency (64 users of 2000 tokens, 16 heads: 98.0 -> 86.3
// us; with three stages 88.4, four CTAs 92.4).
template <int D>
constexpr int dec_ctas() { return D == 64 ? 3 : 2; }
template <int D>
constexpr int dec_stages() { return D == 64 ? 2 : 3; }
constexpr int kDecMaxSms = 160;            // workspace slots: two per CTA

struct AttnDecodeArgs {
  const uint16_t* q;        // [B, Hq, D], rows q_stride apart
  const uint16_t* k_pages;  // [n_pages, Hkv, page_size, D]
  const uint16_t* v_pages;
  KvTables kv;
  const int32_t* slots;     // [B] or null: row b reads slot b
  uint16_t* y;              // [B, Hq, D], rows y_stride apart
  float* lse;               // [B, Hq] or null
  int64_t q_stride, y_stride;
  int B, Hq, Hkv, group;    // group = Hq / Hkv
  int hb, rows;             // head blocks per key-value head, query heads per block (<= 16)
  float scale_log2;         // scale * log2(e)
  float* part;              // [2 G, rows, D] unnormalised outputs
  float* part_ml;           // [2 G, rows, 2] maxima (log2 units) and sums
  int64_t* first_unit;      // [B + 1]
};

// Tokens of batch row b; bad slots and lengths count as empty and are
// recorded by the caller's choice.
__device__ __forceinline__ int decode_len(const AttnDecodeArgs& a, int b, int& slot, bool record) {
  slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.kv.n_slots) {
    if (record) record_error(BITNET_ERR_PAGES);
    slot = 0;
    return 0;
  }
  const int n = a.kv.lens[slot];
  if (n < 0 || (int64_t)n > (int64_t)a.kv.max_pages * a.kv.page_size) {
    if (record) record_error(BITNET_ERR_PAGES);
    return 0;
  }
  return n;
}

// A position in the numbering of units: token block `chunk` of head block vh
// (of Hkv * hb) of batch row b.
struct UnitCursor {
  int b, vh, chunk, chunks, len, slot;
  __device__ __forceinline__ void load_row(const AttnDecodeArgs& a) {
    len = decode_len(a, b, slot, false);
    chunks = (len + kDecUnit - 1) / kDecUnit;
  }
  __device__ __forceinline__ void next(const AttnDecodeArgs& a) {
    if (++chunk < chunks) return;
    chunk = 0;
    if (++vh < a.Hkv * a.hb) return;
    vh = 0;
    do {
      if (++b >= a.B) return;
      load_row(a);
    } while (chunks == 0);
  }
};

template <int D>
constexpr int dec_stage_bytes() { return 2 * 16 * D * 2; }   // 16 keys and values
template <int D, int NT>
constexpr int dec_smem_bytes() {
  return kDecWarps * dec_stages<D>() * dec_stage_bytes<D>() + 2 * 8 * NT * (D + 4) * 4;
}

template <int D, int NT>
__global__ void __launch_bounds__(kDecWarps * 32, dec_ctas<D>()) attn_decode_kernel(const AttnDecodeArgs a) {
  extern __shared__ __align__(128) uint8_t dsm[];
  __shared__ long long s_scan[kDecWarps + 1];
  __shared__ int s_start[3];
  __shared__ float s_ml[2][kDecWarps][16];
  constexpr int kStage = dec_stage_bytes<D>(), kDecStages = dec_stages<D>();
  constexpr int CH = D / 8;                  // 16-byte chunks per row
  constexpr int KT = D / 16;                 // 16-wide steps over D
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* merge = reinterpret_cast<float*>(dsm + kDecWarps * kDecStages * kStage);
  pdl_wait();
  pdl_launch_dependents();

  // ---- the units of all sequences, and this CTA's run of them
  const int VH = a.Hkv * a.hb;
  const int per = (a.B + blockDim.x - 1) / blockDim.x;
  const int b_lo = min(a.B, tid * per), b_hi = min(a.B, b_lo + per);
  long long mine = 0;
  int slot_;
  for (int b = b_lo; b < b_hi; ++b)
    mine += (long long)VH * ((decode_len(a, b, slot_, blockIdx.x == 0) + kDecUnit - 1) / kDecUnit);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  long long before = inc - mine, W = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += s_scan[w];
    W += s_scan[w];
  }
  const long long G = min((long long)gridDim.x, W);      // CTAs with work
  const long long u0 = (int64_t)blockIdx.x < G ? W * blockIdx.x / G : W;
  const long long u1 = (int64_t)blockIdx.x < G ? W * (blockIdx.x + 1) / G : W;
  if (blockIdx.x == 0) {                     // for the joining kernel
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      a.first_unit[b] = at;
      at += (long long)VH * ((decode_len(a, b, slot_, false) + kDecUnit - 1) / kDecUnit);
    }
    if (tid == 0) a.first_unit[a.B] = W;
  }
  if (u0 >= u1) return;                      // the whole block
  if (before <= u0 && u0 < before + mine) {
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const int n = (decode_len(a, b, slot_, false) + kDecUnit - 1) / kDecUnit;
      if (u0 < at + (long long)VH * n) {
        s_start[0] = b;
        s_start[1] = (int)((u0 - at) / n);
        s_start[2] = (int)((u0 - at) % n);
        break;
      }
      at += (long long)VH * n;
    }
  }
  __syncthreads();
  UnitCursor cur;                            // the unit being computed
  cur.b = s_start[0];
  cur.vh = s_start[1];
  cur.chunk = s_start[2];
  cur.load_row(a);
  UnitCursor ld = cur;                       // the unit being loaded
  const int units = (int)(u1 - u0);

  const uint32_t ring = smem_u32(dsm) + (uint32_t)(warp * kDecStages * kStage);
  int loaded = 0;
  uint32_t bad = 0;                          // bit s: stage s holds no page's tokens
  // The page of this warp's tokens in the load cursor's unit is looked up one
  // unit ahead, so that no copy waits for the table.
  int ld_page = -1, ld_row = 0;
  auto look_up = [&]() {
    const int pos = ld.chunk * kDecUnit + warp * 16;
    ld_page = -1;
    if (loaded < units && pos < ld.len) {
      const int e = pos / a.kv.page_size;
      ld_row = pos - e * a.kv.page_size;
      ld_page = a.kv.table[(int64_t)ld.slot * a.kv.max_pages + e];
    }
  };
  look_up();
  // Request this warp's 16 tokens of the load cursor's unit.  Rows behind the
  // sequence's end and pages outside the pool are zero in shared memory (and
  // masked below), so nothing the cache holds there can reach a sum.
  auto load = [&]() {
    if (loaded < units) {
      const int pos = ld.chunk * kDecUnit + warp * 16;
      const int kvh = a.hb == 1 ? ld.vh : ld.vh / a.hb;
      const bool no_page = ld_page < 0 || ld_page >= a.kv.n_pages;
      if (no_page && pos < ld.len && lane == 0) record_error(BITNET_ERR_PAGES);
      const int left = no_page ? 0 : ld.len - pos;
      const uint32_t bit = 1u << (loaded % kDecStages);
      bad = no_page ? bad | bit : bad & ~bit;
      const int64_t off = no_page ? 0
                                  : (((int64_t)ld_page * a.Hkv + kvh) * a.kv.page_size + ld_row) * D;
      const uint32_t dst = ring + (uint32_t)((loaded % kDecStages) * kStage);
      const uint8_t* ks = reinterpret_cast<const uint8_t*>(a.k_pages + off);
      const uint8_t* vs = reinterpret_cast<const uint8_t*>(a.v_pages + off);
#pragma unroll
      for (int i = 0; i < 16 * CH / 32; ++i) {
        const int x = i * 32 + lane, r = x / CH, c = x % CH;
        const uint32_t o = tile_addr<D>(0, r, c);
        const uint32_t n = r < left ? 16u : 0u;
        cp_async16(dst + o, ks + (n ? x * 16 : 0), n);
        cp_async16(dst + 16 * D * 2 + o, vs + (n ? x * 16 : 0), n);
      }
      ld.next(a);
    }
    ++loaded;
    look_up();
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kDecStages - 1; ++i) load();

  uint32_t qf[NT][KT][2];                    // Q^T, the B operand
  float o[KT][NT][4];                        // O^T
  float m[NT][2], l[NT][2];                  // of heads 2 (lane % 4) + {0, 1} of each 8
  bool first_piece = true;
  bool fresh = true;                         // at the start of a piece
  for (int u = 0; u < units; ++u) {
    const int kvh = a.hb == 1 ? cur.vh : cur.vh / a.hb, hblk = cur.vh - kvh * a.hb;
    const int heads = min(a.rows, a.group - hblk * a.rows);
    const int head0 = kvh * a.group + hblk * a.rows;
    if (fresh) {
      fresh = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + (lane >> 2);
        const bool ok = h < heads;
        const uint16_t* qr = a.q + (int64_t)cur.b * a.q_stride + (int64_t)(head0 + (ok ? h : 0)) * D;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const uint32_t* p = reinterpret_cast<const uint32_t*>(qr + kt * 16 + 2 * (lane & 3));
          qf[nt][kt][0] = ok ? p[0] : 0u;
          qf[nt][kt][1] = ok ? p[4] : 0u;
        }
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[kt][nt][i] = 0.f;
      }
    }
    load();
    cp_async_wait<kDecStages - 1>();
    __syncwarp();
    const uint32_t kt_s = ring + (uint32_t)((u % kDecStages) * kStage);
    const uint32_t vt_s = kt_s + 16 * D * 2;
    // S^T = K Q^T: rows are tokens, columns heads
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
    const int mi = lane >> 3;                // matrix of ldmatrix.x4 this lane addresses
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      uint32_t af[4];
      ldsm_x4(tile_addr<D>(kt_s, (lane & 7) + (mi & 1) * 8, kt * 2 + (mi >> 1)), af);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16(s[nt], af, qf[nt][kt][0], qf[nt][kt][1]);
    }
    // tokens past the end, or on no page, are masked
    const int left = (bad >> (u % kDecStages)) & 1u
                         ? 0 : cur.len - (cur.chunk * kDecUnit + warp * 16);
    uint32_t pf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = lane >> 2;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[nt][i] = (i < 2 ? r : r + 8) < left ? s[nt][i] * a.scale_log2 : -INFINITY;
      float t0 = fmaxf(s[nt][0], s[nt][2]), t1 = fmaxf(s[nt][1], s[nt][3]);
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
      }
      t0 = fmaxf(t0, m[nt][0]);
      t1 = fmaxf(t1, m[nt][1]);
      if (__any_sync(0xffffffffu, t0 != m[nt][0] || t1 != m[nt][1])) {
        // a maximum grew: rescale (from -inf, nothing is held yet)
        const float f0 = m[nt][0] == t0 ? 1.f : ex2(m[nt][0] - t0);
        const float f1 = m[nt][1] == t1 ? 1.f : ex2(m[nt][1] - t1);
        l[nt][0] *= f0;
        l[nt][1] *= f1;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          o[kt][nt][0] *= f0;
          o[kt][nt][1] *= f1;
          o[kt][nt][2] *= f0;
          o[kt][nt][3] *= f1;
        }
        m[nt][0] = t0;
        m[nt][1] = t1;
      }
      const float z0 = t0 == -INFINITY ? 0.f : t0, z1 = t1 == -INFINITY ? 0.f : t1;
      const float p0 = ex2(s[nt][0] - z0), p1 = ex2(s[nt][1] - z1);
      const float p2 = ex2(s[nt][2] - z0), p3 = ex2(s[nt][3] - z1);
      l[nt][0] += p0 + p2;
      l[nt][1] += p1 + p3;
      pf[nt][0] = movmatrix_trans(pack_bf16(p0, p1));
      pf[nt][1] = movmatrix_trans(pack_bf16(p2, p3));
    }
    // O^T += V^T P^T
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      uint32_t af[4];
      ldsm_x4_trans(tile_addr<D>(vt_s, (lane & 7) + (mi >> 1) * 8, kt * 2 + (mi & 1)), af);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16(o[kt][nt], af, pf[nt][0], pf[nt][1]);
    }
    __syncwarp();                            // the stage may be refilled

    // ---- end of a piece: join the warps
    UnitCursor nx = cur;
    nx.next(a);
    const bool row_ends = nx.b != cur.b || nx.vh != cur.vh;
    if (row_ends || u + 1 == units) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x);
          if (lane < 4) {
            s_ml[0][warp][nt * 8 + 2 * lane + i] = m[nt][i];
            s_ml[1][warp][nt * 8 + 2 * lane + i] = l[nt][i];
          }
        }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = nt * 8 + 2 * (lane & 3) + i;
          float top = s_ml[0][0][h];
#pragma unroll
          for (int w = 1; w < kDecWarps; ++w) top = fmaxf(top, s_ml[0][w][h]);
          const float f = m[nt][i] == top ? 1.f : ex2(m[nt][i] - top);
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            o[kt][nt][i] *= f;
            o[kt][nt][i + 2] *= f;
          }
        }
      // warps 2 and 3 hand over to 0 and 1, the block adds those two
      float* buf = merge + (warp & 1) * 8 * NT * (D + 4);
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        if ((warp >> 1) == 1 - step) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float* w = buf + (nt * 8 + 2 * (lane & 3) + (i & 1)) * (D + 4) + kt * 16 +
                           (lane >> 2) + (i >> 1) * 8;
                *w = step ? *w + o[kt][nt][i] : o[kt][nt][i];
              }
        }
        __syncthreads();
      }
      const bool whole = row_ends && (!first_piece || s_start[2] == 0);
      const int64_t ps = 2 * (int64_t)blockIdx.x + (first_piece ? 0 : 1);
      for (int x = tid; x < heads * (D / 2); x += blockDim.x) {
        const int h = x / (D / 2), d = 2 * (x % (D / 2));
        float top = s_ml[0][0][h], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kDecWarps; ++w) top = fmaxf(top, s_ml[0][w][h]);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float mw = s_ml[0][w][h];
          sum += mw == top ? s_ml[1][w][h] : s_ml[1][w][h] * ex2(mw - top);
        }
        const float* w0 = merge + h * (D + 4) + d;
        const float* w1 = w0 + 8 * NT * (D + 4);
        const float x0 = w0[0] + w1[0], x1 = w0[1] + w1[1];
        if (whole) {
          // no weight (all scores -inf): 0, whatever the values are
          const float inv = 1.f / sum;
          *reinterpret_cast<uint32_t*>(a.y + (int64_t)cur.b * a.y_stride + (int64_t)(head0 + h) * D +
                                       d) = sum == 0.f ? 0u : pack_bf16(x0 * inv, x1 * inv);
          if (a.lse && d == 0)
            a.lse[(int64_t)cur.b * a.Hq + head0 + h] =
                sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float2*>(a.part + (ps * a.rows + h) * D + d) = make_float2(x0, x1);
          if (d == 0)
            *reinterpret_cast<float2*>(a.part_ml + (ps * a.rows + h) * 2) = make_float2(top, sum);
        }
      }
      __syncthreads();                       // the merge area is free again
      first_piece = false;
      fresh = true;
    }
    cur = nx;
  }
  cp_async_wait<0>();
}

// Joins the pieces of (sequence, head) pairs that several CTAs shared, in the
// order of their units, and writes the rows of empty sequences (0, and -inf
// for the log-sum).  SPLIT warps per query head: the pieces are dealt to them
// in turn, each takes up to 32 at a time (a lane has one piece's maximum and
// sum, a column set per lane for the outputs), and with four warps the last
// step is over shared memory.  Four warps where there are few heads, which
// then have many pieces: 64 heads of 37 pieces took 28 us with one warp each
// and a division per piece.
template <int D, int SPLIT>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnDecodeArgs a, int ctas) {
  constexpr int V = D / 32;                  // outputs per lane
  __shared__ float s_acc[SPLIT][D], s_ml[SPLIT][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = SPLIT == 1 ? 0 : warp;
  const int64_t id = SPLIT == 1 ? (int64_t)blockIdx.x * 4 + warp : (int64_t)blockIdx.x;
  pdl_wait();
  if (id >= (int64_t)a.B * a.Hq) return;
  const int b = (int)(id / a.Hq), head = (int)(id % a.Hq);
  uint16_t* yr = a.y + (int64_t)b * a.y_stride + (int64_t)head * D + lane * V;
  const long long W = a.first_unit[a.B], at = a.first_unit[b], to = a.first_unit[b + 1];
  const int chunks = (int)((to - at) / ((long long)a.Hkv * a.hb));
  if (chunks == 0) {
    if (part == 0) {
#pragma unroll
      for (int i = 0; i < V; i += 2) *reinterpret_cast<uint32_t*>(yr + i) = 0u;
      if (a.lse && lane == 0) a.lse[id] = -INFINITY;
    }
    return;
  }
  const long long G = min((long long)ctas, W);
  const int kvh = head / a.group, in_group = head % a.group;
  const int vh = kvh * a.hb + in_group / a.rows, row = in_group % a.rows;
  const long long ua = at + (long long)vh * chunks;
  const int c0 = (int)(((ua + 1) * G - 1) / W), c1 = (int)(((ua + chunks) * G - 1) / W);
  if (c0 == c1) return;                      // finished by its CTA
  // CTA c0 holds its piece as its last one unless it starts with it, the
  // others as their first one
  const int first_slot = W * c0 / G == ua ? 2 * c0 : 2 * c0 + 1;
  float top = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int p0 = part; p0 <= c1 - c0; p0 += 32 * SPLIT) {
    const int p = p0 + lane * SPLIT;
    const int slot = p == 0 ? first_slot : 2 * (c0 + p);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (p <= c1 - c0)
      ml = *reinterpret_cast<const float2*>(a.part_ml + ((int64_t)slot * a.rows + row) * 2);
    const float t = fmaxf(top, warp_max(ml.x));
    const float f0 = top == t ? 1.f : ex2(top - t), f = ml.x == t ? 1.f : ex2(ml.x - t);
    top = t;
    sum = sum * f0 + f * ml.y;               // per lane until the end
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= f0;
    const int n = min(32, (c1 - c0 - p0) / SPLIT + 1);
#pragma unroll 8
    for (int x = 0; x < n; ++x) {
      const float fx = __shfl_sync(0xffffffffu, f, x);
      const int sx = __shfl_sync(0xffffffffu, slot, x);
      const float* w = a.part + ((int64_t)sx * a.rows + row) * D + lane * V;
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 v = *reinterpret_cast<const float2*>(w + i);
        acc[i] += fx * v.x;
        acc[i + 1] += fx * v.y;
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (SPLIT > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) s_acc[part][lane * V + i] = acc[i];
    if (lane == 0) {
      s_ml[part][0] = top;
      s_ml[part][1] = sum;
    }
    __syncthreads();
    if (part != 0) return;
    float all = s_ml[0][0];
#pragma unroll
    for (int w = 1; w < SPLIT; ++w) all = fmaxf(all, s_ml[w][0]);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < SPLIT; ++w) {
      const float f = s_ml[w][0] == all ? 1.f : ex2(s_ml[w][0] - all);
      sum += f * s_ml[w][1];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += f * s_acc[w][lane * V + i];
    }
    top = all;
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(yr + i) =
        sum == 0.f ? 0u : pack_bf16(acc[i] * inv, acc[i + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[id] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace bitnet
