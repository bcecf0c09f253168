// C ABI of the attention and key-value cache operators: argument validation
// and launches.  Contracts are in include/bitnet.h.
#include <cmath>

#include "attention.cuh"

using namespace bitnet;

namespace {

constexpr int64_t kMaxI32 = 0x7fffffff;
constexpr double kLog2e = 1.4426950408889634;

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool ranges_overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Launch with programmatic dependent launch (every kernel here begins with
// griddepcontrol.wait).
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                       cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The checks every call with tables shares.
bitnet_status check_tables(const bitnet_kv_tables* kv) {
  if (!kv || !kv->table || !kv->lens || !kv->refs) return BITNET_ERR_INVALID_ARG;
  if (kv->n_slots < 1 || kv->n_slots > kKvMaxSlots || kv->max_pages < 1 || kv->n_pages < 1 ||
      kv->n_pages > (1 << 30) || kv->page_size < 16 || kv->page_size > 1024 ||
      kv->page_size % 16 != 0 || kv->max_pages > kMaxI32 / 2 / kv->page_size)
    return BITNET_ERR_SHAPE;
  if (!aligned4(kv->table) || !aligned4(kv->lens) || !aligned4(kv->refs)) return BITNET_ERR_ALIGN;
  return BITNET_OK;
}

KvTables device_tables(const bitnet_kv_tables* kv) {
  KvTables t{};
  t.table = kv->table;
  t.lens = kv->lens;
  t.refs = kv->refs;
  t.n_slots = (int)kv->n_slots;
  t.max_pages = (int)kv->max_pages;
  t.n_pages = (int)kv->n_pages;
  t.page_size = (int)kv->page_size;
  return t;
}

bool heads_ok(int64_t Hq, int64_t Hkv, int64_t D) {
  return (D == 64 || D == 128) && Hkv >= 1 && Hq >= Hkv && Hq <= 65536 && Hq % Hkv == 0 &&
         Hq / Hkv <= 64;
}
// A scale whose product with log2 e, by which the kernels multiply, is a number.
bool scale_ok(float scale) {
  return scale > 0.0f && std::isfinite((float)((double)scale * kLog2e));
}
bool stride_ok(int64_t stride, int64_t width) {
  return stride >= width && stride % 8 == 0 && stride <= kMaxI32;
}

// The decode kernel's workspace: partial outputs, their maxima and sums, the
// first unit of every row.
struct DecodeWs {
  int hb, rows;
  size_t part, ml, first, total;
};
DecodeWs decode_ws(int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  DecodeWs w{};
  const int g = (int)(Hq / Hkv);
  w.hb = (g + 15) / 16;
  w.rows = (g + w.hb - 1) / w.hb;
  const size_t n = (size_t)2 * kDecMaxSms * (D == 64 ? dec_ctas<64>() : dec_ctas<128>()) * w.rows;
  w.part = 0;
  w.ml = al256(n * D * 4);
  w.first = w.ml + al256(n * 8);
  w.total = w.first + al256((size_t)(B + 1) * 8);
  return w;
}

template <int D, int NT>
bitnet_status decode_launch(const AttnDecodeArgs& a, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  constexpr int smem = dec_smem_bytes<D, NT>();
  if (set_smem_attr_once(configured, attn_decode_kernel<D, NT>, smem) != cudaSuccess)
    return BITNET_ERR_CUDA;
  if (launch_pdl(attn_decode_kernel<D, NT>, (unsigned)ctas, kDecWarps * 32, smem, s, a) !=
      cudaSuccess)
    return BITNET_ERR_CUDA;
  const int64_t heads = (int64_t)a.B * a.Hq;
  const cudaError_t e =
      heads <= 4 * ctas
          ? launch_pdl(attn_join_kernel<D, 4>, (unsigned)heads, 128, 0, s, a, ctas)
          : launch_pdl(attn_join_kernel<D, 1>, (unsigned)((heads + 3) / 4), 128, 0, s, a, ctas);
  if (e != cudaSuccess) return BITNET_ERR_CUDA;
  return BITNET_OK;
}

// Upper bound of the tiles of `tokens` tokens (the lengths are on the device).
int64_t prompt_ctas(const AttnPromptArgs& a, int tokens) {
  return ((int64_t)(a.Tq / tokens) + a.B) * a.Hkv;
}

template <int D>
bitnet_status prompt_warp_launch(AttnPromptArgs a, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  constexpr int smem = pw_smem_bytes<D>();
  if (set_smem_attr_once(configured, prompt_warp_kernel<D>, smem) != cudaSuccess)
    return BITNET_ERR_CUDA;
  a.tile_tokens = kPwRows / a.group;
  const int64_t grid = prompt_ctas(a, a.tile_tokens);
  if (grid > kMaxI32) return BITNET_ERR_SHAPE;
  return launch_pdl(prompt_warp_kernel<D>, (unsigned)grid, 128, smem, s, a) == cudaSuccess
             ? BITNET_OK : BITNET_ERR_CUDA;
}

// Tokens by heads by D: a map whose boxes are 64 columns of `heads` heads of
// `tokens` tokens, 128-byte swizzled.
bool make_map_tokens(CUtensorMap* m, const void* base, int64_t D, int64_t H, int64_t T,
                     int64_t stride, uint32_t heads, uint32_t tokens) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, heads, tokens}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
bitnet_status prompt_tile_launch(AttnPromptArgs a, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  constexpr size_t smem = PtCfg<D>::kSmem;
  // The kernel's softmax warps ask for kPtRegs registers; a build that launches
  // it with fewer would have them wait for registers that no warp gives back.
  static const bool regs_ok = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, prompt_tile_kernel<D>) == cudaSuccess && f.numRegs >= kPtRegs;
  }();
  if (!regs_ok) return BITNET_ERR_UNSUPPORTED;
  if (set_smem_attr_once(configured, prompt_tile_kernel<D>, (int)smem) != cudaSuccess)
    return BITNET_ERR_CUDA;
  const int half = 128 / a.group;
  a.half_tokens = half;
  a.tile_tokens = 2 * half;
  int64_t grid = prompt_ctas(a, a.tile_tokens);
  // Too few tiles for the SMs: tiles of one half each, twice as many.  A step
  // of one half takes about 0.7 of the time of two, with D = 64 (bound by the
  // exponentials) less.  One wave of halves: 512 / 1024 tokens of 20 heads 13.4 /
  // 20.0 -> 10.6 / 16.0 us, 200 rows on 8000 keys 115 -> 83.  More than one wave
  // pays with D = 64 (1000 rows on 5000 keys of 16 heads 69 -> 56 us, 2048 tokens
  // 32 -> 28) and not with D = 128 (512 rows on 4096 keys of 64 heads 64 -> 86,
  // 512 tokens of 64 heads 14.1 -> 18.4).
  if (prompt_ctas(a, half) <= num_sms || (D == 64 && grid <= num_sms)) {
    a.tile_tokens = half;
    grid = prompt_ctas(a, half);
  }
  if (grid > kMaxI32) return BITNET_ERR_SHAPE;
  CUtensorMap tq, tk, tv;
  if (!make_map_tokens(&tq, a.q, D, a.Hq, a.Tq, a.q_stride, (uint32_t)a.group, (uint32_t)half) ||
      !make_map_tokens(&tk, a.k, D, a.Hkv, a.Tk, a.k_stride, 1, kPtKeys) ||
      !make_map_tokens(&tv, a.v, D, a.Hkv, a.Tk, a.v_stride, 1, kPtKeys))
    return BITNET_ERR_CUDA;
  return launch_pdl(prompt_tile_kernel<D>, (unsigned)grid, kPtThreads, smem, s, tq, tk, tv, a) ==
                 cudaSuccess
             ? BITNET_OK : BITNET_ERR_CUDA;
}

unsigned kv_blocks(int64_t items, int num_sms) {
  const int64_t b = (items + 255) / 256;
  return (unsigned)(b < (int64_t)num_sms * 8 ? b : (int64_t)num_sms * 8);
}

}  // namespace

extern "C" {

bitnet_status bitnet_attn_prompt(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                 int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                 const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t Tq,
                                 int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, float scale,
                                 uint16_t* y, int64_t y_stride, float* lse, void* stream) {
  if (!q || !k || !v || !cu_q || !cu_k || !y) return BITNET_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return BITNET_ERR_INVALID_ARG;
  if (B < 1 || B > kMaxI32 / 2 || Tq < 1 || Tq > kMaxI32 / 2 || Tk < 1 || Tk > kMaxI32 / 2 ||
      !heads_ok(Hq, Hkv, D) || !stride_ok(q_stride, Hq * D) || !stride_ok(y_stride, Hq * D) ||
      !stride_ok(k_stride, Hkv * D) || !stride_ok(v_stride, Hkv * D))
    return BITNET_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(y) || !aligned4(cu_q) ||
      !aligned4(cu_k) || !aligned4(lse))
    return BITNET_ERR_ALIGN;
  const int64_t yb = ((Tq - 1) * y_stride + Hq * D) * 2;
  if (ranges_overlap(y, yb, q, ((Tq - 1) * q_stride + Hq * D) * 2) ||
      ranges_overlap(y, yb, k, ((Tk - 1) * k_stride + Hkv * D) * 2) ||
      ranges_overlap(y, yb, v, ((Tk - 1) * v_stride + Hkv * D) * 2))
    return BITNET_ERR_INVALID_ARG;
  DevInfo d;
  const bitnet_status st = device_info(&d);
  if (st != BITNET_OK) return st;
  AttnPromptArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.cu_q = cu_q; a.cu_k = cu_k;
  a.y = y; a.lse = lse;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.y_stride = y_stride;
  a.B = (int)B; a.Tq = (int)Tq; a.Tk = (int)Tk;
  a.Hq = (int)Hq; a.Hkv = (int)Hkv; a.group = (int)(Hq / Hkv);
  a.scale = scale;
  a.scale_log2 = (float)((double)scale * kLog2e);
  // Very short prompts, few of them: the warp kernel starts faster (no tensor
  // memory, no tensor maps).  20 heads of 128, one prompt of 32 / 64 / 96 / 192
  // tokens: 6.1 / 6.3 / 7.5 / 9.0 us against the tile kernel's 6.3 / 6.4 / 7.1 /
  // 7.6; 16 heads of 64, 64 / 128 / 192 / 256 tokens: 4.5 / 5.4 / 6.4 / 7.3 against
  // 5.5 / 6.2 / 6.3 / 7.0.  The lengths are on the device, so several sequences
  // may be one long one and empty ones: the sum is held where that costs less
  // than equal lengths gain.  20 sequences of 128 tokens in all, 12 heads of 128:
  // equal 5.8 against 6.6, one of 128 7.4 against 6.8 (of 512: 6.2 / 7.0, 16.1 /
  // 10.5); of 256 in all, 8 heads of 64: 4.7 / 5.8 and 7.6 / 7.1 (of 768: 4.7 / 5.7,
  // 15.4 / 11.6).
  const int64_t each = D == 64 ? 192 : 64, all = D == 64 ? 256 : 128;
  const bool few = prompt_ctas(a, kPwRows / a.group) * 2 <= 3 * d.num_sms && Tk <= all &&
                   Tk <= each * B;
  if (few)
    return D == 64 ? prompt_warp_launch<64>(a, as_stream(stream))
                   : prompt_warp_launch<128>(a, as_stream(stream));
  return D == 64 ? prompt_tile_launch<64>(a, d.num_sms, as_stream(stream))
                 : prompt_tile_launch<128>(a, d.num_sms, as_stream(stream));
}

size_t bitnet_attn_decode_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B < 1 || B > kKvMaxSlots || !heads_ok(Hq, Hkv, D)) return 0;
  return decode_ws(B, Hq, Hkv, D).total;
}

bitnet_status bitnet_attn_decode(const uint16_t* q, int64_t q_stride, const uint16_t* k_pages,
                                 const uint16_t* v_pages, const bitnet_kv_tables* kv,
                                 const int32_t* slots, int64_t B, int64_t Hq, int64_t Hkv,
                                 int64_t D, float scale, uint16_t* y, int64_t y_stride,
                                 float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!q || !k_pages || !v_pages || !y) return BITNET_ERR_INVALID_ARG;
  bitnet_status st = check_tables(kv);
  if (st != BITNET_OK) return st;
  if (!scale_ok(scale)) return BITNET_ERR_INVALID_ARG;
  if (B < 1 || B > kKvMaxSlots || (!slots && B > kv->n_slots) || !heads_ok(Hq, Hkv, D) ||
      !stride_ok(q_stride, Hq * D) || !stride_ok(y_stride, Hq * D))
    return BITNET_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(y) ||
      !aligned4(slots) || !aligned4(lse))
    return BITNET_ERR_ALIGN;
  const int64_t yb = ((B - 1) * y_stride + Hq * D) * 2;
  const int64_t cb = kv->n_pages * Hkv * kv->page_size * D * 2;
  if (ranges_overlap(y, yb, q, ((B - 1) * q_stride + Hq * D) * 2) ||
      ranges_overlap(y, yb, k_pages, cb) || ranges_overlap(y, yb, v_pages, cb))
    return BITNET_ERR_INVALID_ARG;
  const DecodeWs w = decode_ws(B, Hq, Hkv, D);
  if (!workspace || workspace_bytes < w.total) return BITNET_ERR_WORKSPACE;
  if (!aligned16(workspace)) return BITNET_ERR_ALIGN;
  DevInfo d;
  st = device_info(&d);
  if (st != BITNET_OK) return st;
  AttnDecodeArgs a{};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.q = q; a.k_pages = k_pages; a.v_pages = v_pages;
  a.kv = device_tables(kv);
  a.slots = slots;
  a.y = y; a.lse = lse;
  a.q_stride = q_stride; a.y_stride = y_stride;
  a.B = (int)B; a.Hq = (int)Hq; a.Hkv = (int)Hkv; a.group = (int)(Hq / Hkv);
  a.hb = w.hb; a.rows = w.rows;
  a.scale_log2 = (float)((double)scale * kLog2e);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float*>(ws + w.ml);
  a.first_unit = reinterpret_cast<int64_t*>(ws + w.first);
  const int ctas = (d.num_sms < kDecMaxSms ? d.num_sms : kDecMaxSms) *
                   (D == 64 ? dec_ctas<64>() : dec_ctas<128>());
  cudaStream_t s = as_stream(stream);
  if (D == 64) return w.rows <= 8 ? decode_launch<64, 1>(a, ctas, s) : decode_launch<64, 2>(a, ctas, s);
  return w.rows <= 8 ? decode_launch<128, 1>(a, ctas, s) : decode_launch<128, 2>(a, ctas, s);
}

size_t bitnet_kv_workspace_size(int64_t n_slots, int64_t n_pages) {
  if (n_slots < 1 || n_slots > kKvMaxSlots || n_pages < 1 || n_pages > (1 << 30)) return 0;
  return al256((size_t)(4 + n_slots + 2 * n_pages) * 4);
}

bitnet_status bitnet_kv_extend(const bitnet_kv_tables* kv, const int32_t* slots,
                               const int32_t* add, int64_t n, int32_t* short_pages,
                               void* workspace, size_t workspace_bytes, void* stream) {
  bitnet_status st = check_tables(kv);
  if (st != BITNET_OK) return st;
  if (!add) return BITNET_ERR_INVALID_ARG;
  if (n < 1 || n > kv->n_slots) return BITNET_ERR_SHAPE;
  if (!aligned4(slots) || !aligned4(add) || !aligned4(short_pages)) return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_kv_workspace_size(kv->n_slots, kv->n_pages))
    return BITNET_ERR_WORKSPACE;
  if (!aligned16(workspace)) return BITNET_ERR_ALIGN;
  DevInfo d;
  st = device_info(&d);
  if (st != BITNET_OK) return st;
  return launch_pdl(kv_extend_kernel, 1, kKvThreads, 0, as_stream(stream), device_tables(kv), slots,
                    add, (int)n, short_pages, static_cast<int32_t*>(workspace)) == cudaSuccess
             ? BITNET_OK : BITNET_ERR_CUDA;
}

bitnet_status bitnet_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                               int64_t v_stride, const int32_t* cu, const int32_t* slots,
                               int64_t B, int64_t T, int64_t Hkv, int64_t D,
                               const bitnet_kv_tables* kv, uint16_t* k_pages, uint16_t* v_pages,
                               void* stream) {
  if (!k || !v || !cu || !k_pages || !v_pages) return BITNET_ERR_INVALID_ARG;
  bitnet_status st = check_tables(kv);
  if (st != BITNET_OK) return st;
  if (B < 1 || B > kKvMaxSlots || (!slots && B > kv->n_slots) || T < 1 || T > kMaxI32 / 2 ||
      !heads_ok(Hkv, Hkv, D) || !stride_ok(k_stride, Hkv * D) || !stride_ok(v_stride, Hkv * D))
    return BITNET_ERR_SHAPE;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) ||
      !aligned4(cu) || !aligned4(slots))
    return BITNET_ERR_ALIGN;
  const int64_t cb = kv->n_pages * Hkv * kv->page_size * D * 2;
  const int64_t kb = ((T - 1) * k_stride + Hkv * D) * 2, vb = ((T - 1) * v_stride + Hkv * D) * 2;
  if (ranges_overlap(k_pages, cb, v_pages, cb) || ranges_overlap(k_pages, cb, k, kb) ||
      ranges_overlap(k_pages, cb, v, vb) || ranges_overlap(v_pages, cb, k, kb) ||
      ranges_overlap(v_pages, cb, v, vb))
    return BITNET_ERR_INVALID_ARG;
  DevInfo d;
  st = device_info(&d);
  if (st != BITNET_OK) return st;
  KvAppendArgs a{};
  a.k = k; a.v = v; a.cu = cu; a.slots = slots;
  a.kv = device_tables(kv);
  a.k_pages = k_pages; a.v_pages = v_pages;
  a.k_stride = k_stride; a.v_stride = v_stride;
  a.B = (int)B; a.T = (int)T; a.Hkv = (int)Hkv;
  return launch_pdl(D == 64 ? kv_append_kernel<64> : kv_append_kernel<128>, (unsigned)((T + 7) / 8), 256, 0, as_stream(stream), a) ==
                 cudaSuccess
             ? BITNET_OK : BITNET_ERR_CUDA;
}

bitnet_status bitnet_kv_fork(const bitnet_kv_tables* kv, const int32_t* parents,
                             const int32_t* children, int64_t n, int32_t* pairs, int32_t* n_pairs,
                             int32_t* short_pages, void* workspace, size_t workspace_bytes,
                             void* stream) {
  bitnet_status st = check_tables(kv);
  if (st != BITNET_OK) return st;
  if (!parents || !children || !pairs || !n_pairs) return BITNET_ERR_INVALID_ARG;
  if (n < 1 || n > kv->n_slots) return BITNET_ERR_SHAPE;
  if (!aligned4(parents) || !aligned4(children) || !aligned4(pairs) || !aligned4(n_pairs) ||
      !aligned4(short_pages))
    return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_kv_workspace_size(kv->n_slots, kv->n_pages))
    return BITNET_ERR_WORKSPACE;
  if (!aligned16(workspace)) return BITNET_ERR_ALIGN;
  DevInfo d;
  st = device_info(&d);
  if (st != BITNET_OK) return st;
  const KvTables t = device_tables(kv);
  int32_t* ws = static_cast<int32_t*>(workspace);
  cudaStream_t s = as_stream(stream);
  const bool one_block = n * kv->max_pages <= kKvOneBlock;
  if (launch_pdl(kv_fork_plan_kernel, 1, kKvThreads, 0, s, t, parents, children, (int)n, pairs,
                 n_pairs, short_pages, ws, one_block) != cudaSuccess)
    return BITNET_ERR_CUDA;
  if (one_block) return BITNET_OK;
  return launch_pdl(kv_fork_rows_kernel, kv_blocks(n * kv->max_pages, d.num_sms), 256, 0, s, t,
                    parents, children, (int)n, (const int32_t*)ws) == cudaSuccess
             ? BITNET_OK : BITNET_ERR_CUDA;
}

bitnet_status bitnet_kv_free(const bitnet_kv_tables* kv, const int32_t* slots, int64_t n,
                             void* stream) {
  bitnet_status st = check_tables(kv);
  if (st != BITNET_OK) return st;
  if (!slots) return BITNET_ERR_INVALID_ARG;
  if (n < 1 || n > kKvMaxSlots) return BITNET_ERR_SHAPE;
  if (!aligned4(slots)) return BITNET_ERR_ALIGN;
  DevInfo d;
  st = device_info(&d);
  if (st != BITNET_OK) return st;
  return launch_pdl(kv_free_kernel, kv_blocks(n * kv->max_pages, d.num_sms), 256, 0,
                    as_stream(stream), device_tables(kv), slots, (int)n) == cudaSuccess
             ? BITNET_OK : BITNET_ERR_CUDA;
}

bitnet_status bitnet_kv_compact(const bitnet_kv_tables* kv, int32_t* pairs, int32_t* n_pairs,
                                int32_t* live, void* workspace, size_t workspace_bytes,
                                void* stream) {
  bitnet_status st = check_tables(kv);
  if (st != BITNET_OK) return st;
  if (!pairs || !n_pairs) return BITNET_ERR_INVALID_ARG;
  if (!aligned4(pairs) || !aligned4(n_pairs) || !aligned4(live)) return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_kv_workspace_size(kv->n_slots, kv->n_pages))
    return BITNET_ERR_WORKSPACE;
  if (!aligned16(workspace)) return BITNET_ERR_ALIGN;
  DevInfo d;
  st = device_info(&d);
  if (st != BITNET_OK) return st;
  const KvTables t = device_tables(kv);
  int32_t* ws = static_cast<int32_t*>(workspace);
  cudaStream_t s = as_stream(stream);
  const bool one_block = kv->n_slots * kv->max_pages <= kKvOneBlock;
  if (launch_pdl(kv_compact_plan_kernel, 1, kKvThreads, 0, s, t, pairs, n_pairs, live, ws,
                 one_block) != cudaSuccess)
    return BITNET_ERR_CUDA;
  if (one_block) return BITNET_OK;
  return launch_pdl(kv_compact_table_kernel, kv_blocks(kv->n_slots * kv->max_pages, d.num_sms), 256,
                    0, s, t, (const int32_t*)ws) == cudaSuccess
             ? BITNET_OK : BITNET_ERR_CUDA;
}

bitnet_status bitnet_kv_copy_pages(int64_t L, uint16_t* const* k_pages, uint16_t* const* v_pages,
                                   int64_t n_pages, int64_t page_bytes, const int32_t* pairs,
                                   const int32_t* n_pairs, int64_t max_pairs, void* stream) {
  if (!k_pages || !v_pages || !pairs || !n_pairs || L < 1) return BITNET_ERR_INVALID_ARG;
  if (n_pages < 1 || n_pages > (1 << 30) || page_bytes < 16 || page_bytes % 16 != 0 ||
      page_bytes > (int64_t(1) << 34) || max_pairs < 1 || max_pairs > n_pages || L > 65536)
    return BITNET_ERR_SHAPE;
  for (int64_t l = 0; l < L; ++l) {
    if (!k_pages[l] || !v_pages[l]) return BITNET_ERR_INVALID_ARG;
    if (!aligned16(k_pages[l]) || !aligned16(v_pages[l])) return BITNET_ERR_ALIGN;
  }
  if (!aligned4(pairs) || !aligned4(n_pairs)) return BITNET_ERR_ALIGN;
  DevInfo d;
  const bitnet_status st = device_info(&d);
  if (st != BITNET_OK) return st;
  for (int64_t l0 = 0; l0 < L; l0 += kCopyLayers) {
    const int layers = (int)(L - l0 < kCopyLayers ? L - l0 : kCopyLayers);
    KvCopyArgs a{};
    for (int l = 0; l < layers; ++l) {
      a.base[2 * l] = reinterpret_cast<uint4*>(k_pages[l0 + l]);
      a.base[2 * l + 1] = reinterpret_cast<uint4*>(v_pages[l0 + l]);
    }
    a.pairs = pairs; a.n_pairs = n_pairs;
    a.max_pairs = (int)max_pairs; a.n_pages = (int)n_pages; a.planes = 2 * layers;
    a.page_chunks = page_bytes / 16;
    if (launch_pdl(kv_copy_kernel, (unsigned)(d.num_sms * 8), kCopyThreads, 0, as_stream(stream),
                   a) != cudaSuccess)
      return BITNET_ERR_CUDA;
  }
  return BITNET_OK;
}

}  // extern "C"
