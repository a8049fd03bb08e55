// What the forward and backward kernels of the attention operator share: the
// arguments, which 128-key (or 128-query) tiles a CTA visits, and the scores'
// cap and distance bias.
#pragma once

#include "op_tma.cuh"

namespace sdo {

constexpr int kTile = 128;                       // query rows and keys per tile
constexpr int kBlockBytes = kTile * 64 * 2;      // 128 rows x 64 head dimensions, swizzled
constexpr int kMaxTiles = (1 << 20) / kTile;     // k_len, q_len <= 2^20
constexpr int kTileWords = kMaxTiles / 32;

struct AttnArgs {
  int32_t B, Nq, Nk, H, KV, G, D;   // G = H / KV query heads per key head
  int32_t tq;                       // forward: query tokens of a tile (kTile / G, all G heads of each)
  int32_t qtiles, ktiles, splits;
  int32_t causal;
  float sl2;                        // scale * log2(e)
  float cap_in, cap_out;            // tanh(s * cap_in) * cap_out = capped score in log2 units; cap_out 0 = no cap
  const int32_t *k_lens, *prefix, *q_doc, *k_doc;
  const float* slopes;
  const int32_t* k_range;           // [B][ktiles][2] lowest and highest document of each key tile
  const int32_t* q_range;           // backward: the same of the 128-query tiles
  int64_t os[3];
  void* o;
  float* lse;
  float* partial;                   // forward split: [items][splits][128][D], then max and sum [items][splits][128][2]
  float* partial_ml;
  int* err;
  int32_t clear_err;
};

// One bit per tile, in shared memory.
struct alignas(16) TileBits {
  uint32_t see[kTileWords];  // some row may see some key of the tile
  uint32_t all[kTileWords];  // every row sees every key
  int32_t count;             // tiles in `see`
};
static_assert(sizeof(TileBits) % 16 == 0, "what follows it in shared memory is read in 16-byte accesses");

// Walks the tiles of `see` in order, from the rank-th on.
struct TileWalk {
  const TileBits* t;
  uint32_t left;  // bits of the current word not yet visited
  int word, words;
  __device__ __forceinline__ void start(const TileBits* bits, int ntiles, int rank) {
    t = bits;
    words = (ntiles + 31) >> 5;
    word = 0;
    left = t->see[0];
    while (word < words - 1) {
      const int n = __popc(left);
      if (rank < n) break;
      rank -= n;
      left = t->see[++word];
    }
    for (; rank > 0; --rank) left &= left - 1;
  }
  // The next tile's index (the caller knows that there is one).
  __device__ __forceinline__ int next() {
    while (left == 0 && word < words - 1) left = t->see[++word];
    const int j = word * 32 + __ffs(left) - 1;
    left &= left - 1;
    return j;
  }
  __device__ __forceinline__ bool whole(int j) const { return (t->all[j >> 5] >> (j & 31)) & 1; }
};

__device__ __forceinline__ int keys_of(const AttnArgs& a, int b) {
  return a.k_lens ? min(max(a.k_lens[b], 0), a.Nk) : a.Nk;
}
__device__ __forceinline__ int prefix_of(const AttnArgs& a, int b) { return a.prefix ? a.prefix[b] : 0; }

// tanh through one exponential and one reciprocal: absolute error near 2^-22, so the
// capped score is off by 2^-22 of the cap (the one-instruction tanh is off by 2^-11).
__device__ __forceinline__ float tanh_acc(float x) {
  return fmaf(-2.f, fast_rcp(1.f + fast_ex2(2.f * kLog2e * x)), 1.f);
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Launches of the backward pass (attention_grad.cu).
struct AttnCall {
  const sd_attention_cfg* cfg;
  int64_t qs[3], ks[3], vs[3], os[3];
  const void *q, *k, *v, *o, *d_o;
  void *dq, *dk, *dv;
  const float* lse;
  AttnArgs args;
  uint8_t* ws;
  Device dev;
  cudaStream_t st;
};
size_t attn_grad_space(const sd_attention_cfg& c);
template <typename T>
sd_status attn_backward(AttnCall& c);
// Map of a [batch][tokens][heads][D] tensor; a box holds box_heads x box_tokens rows of 64.
bool attn_map(CUtensorMap* m, bool f16, const void* p, const int64_t* s, int batch, int tokens, int heads, int d,
              uint32_t box_heads, uint32_t box_tokens);
// Lowest and highest document id of each 128-token tile.
sd_status attn_doc_ranges(const int32_t* doc, int batch, int len, int32_t* range, cudaStream_t st);
void attn_fill(AttnCall& c, const sd_attention_masks* m);

}  // namespace sdo
