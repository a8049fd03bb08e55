// What the forward and backward kernels of the attention operator share: the
// arguments, which 128-key (or 128-query) tiles a CTA visits, and the scores'
// cap and distance bias.
#pragma once

#include <string.h>

#include "op_tma.cuh"

namespace sdo {

constexpr int kTile = 128;                       // query rows and keys per tile
constexpr int kBlockBytes = kTile * 64 * 2;      // 128 rows x 64 head dimensions, swizzled

// How items of work (query tiles, key tiles) are cut into units: groups of consecutive
// items, each item of a group into the same number of parts. Parts of cut items have
// slots in the scratch, in unit order; cut items are consecutive over the groups.
constexpr int kGroups = 8;
struct Parts {
  int32_t n;               // groups
  int32_t item[kGroups];   // first item of each
  int32_t unit[kGroups];   // first unit
  int32_t parts[kGroups];  // of an item
  int32_t slot[kGroups];   // first slot, where parts > 1
  int32_t first, count;    // the cut items
  __device__ __forceinline__ int group_of_item(int i) const {
    int g = 0;
    while (g + 1 < n && i >= item[g + 1]) ++g;
    return g;
  }
};
// Part z of `parts` of an item; its slot, or -1 where the item is not cut.
struct Part {
  int item, z, parts, slot;
  __device__ __forceinline__ Part(const Parts& p, int u) {
    int g = 0;
    while (g + 1 < p.n && u >= p.unit[g + 1]) ++g;
    parts = p.parts[g];
    const int at = u - p.unit[g];
    item = p.item[g] + at;
    z = 0;
    slot = -1;
    if (parts > 1) {
      item = p.item[g] + at / parts;
      z = at % parts;
      slot = p.slot[g] + at;
    }
  }
  // the first of `count` steps that are this part's, and how many
  __device__ __forceinline__ int64_t begin(int64_t count) const { return count * z / parts; }
  __device__ __forceinline__ int steps(int64_t count) const {
    return (int)(count * (z + 1) / parts - begin(count));
  }
};

struct AttnArgs {
  int32_t B, Nq, Nk, H, KV, G, D;   // G = H / KV query heads per key head
  int32_t tq;                       // forward: query tokens of a tile (kTile / G, all G heads of each)
  int32_t qtiles, ktiles;
  Parts parts;                      // forward: items are query tiles x key heads x sequences
  int32_t causal;
  float sl2;                        // scale * log2(e)
  float cap_in, cap_out;            // tanh(s * cap_in) * cap_out = capped score in log2 units; cap_out 0 = no cap
  const int32_t *k_lens, *prefix, *q_doc, *k_doc;
  const float* slopes;
  const int32_t* k_range;           // [B][ktiles][2] lowest and highest document of each key tile
  const int32_t* q_range;           // the same of the query tiles (tq tokens forward, 128 backward)
  const int32_t *k_pad, *q_pad;     // the documents again, rows of whole 128-token tiles
  int64_t os[3];
  void* o;
  float* lse;
  float* partial;                   // forward: [slots][128][D], then max and sum [slots][128][2]
  float* partial_ml;
  int* err;
  int32_t clear_err;
  int32_t hold_spins;               // tests only: the loading warp first waits, this long, for what never comes
};

__device__ __forceinline__ int keys_of(const AttnArgs& a, int b) {
  return a.k_lens ? min(max(a.k_lens[b], 0), a.Nk) : a.Nk;
}
__device__ __forceinline__ int prefix_of(const AttnArgs& a, int b) { return a.prefix ? max(a.prefix[b], 0) : 0; }

// Which key tiles 128 query rows (tokens i0 .. i1 of sequence b) may see: those
// before lim_any whose documents meet [lo, hi]; every row sees all of the tiles
// before lim_all that hold the one document lo = hi.
struct RowTiles {
  const int32_t* range;  // documents of the key tiles, or null
  int lim_any, lim_all, lo, hi;
  __device__ __forceinline__ RowTiles(const AttnArgs& a, int b, int i0, int i1, int off, int nk, int pre,
                                      const int32_t* q_range) {
    lim_any = a.causal ? min(nk, max(i1 + off + 1, pre)) : nk;
    lim_all = a.causal ? min(nk, max(i0 + off + 1, pre)) : nk;
    range = a.k_range ? a.k_range + (int64_t)b * a.ktiles * 2 : nullptr;
    lo = range ? q_range[0] : 0;
    hi = range ? q_range[1] : 0;
  }
  __device__ __forceinline__ int tiles() const { return (lim_any + kTile - 1) / kTile; }
  __device__ __forceinline__ void look(int j, bool& see, bool& all) const {
    see = j * kTile < lim_any;
    all = (j + 1) * kTile <= lim_all;
    if (see && range) {
      const int32_t l = range[2 * j], h = range[2 * j + 1];
      see = l <= hi && lo <= h;
      all = all && l == h && lo == l && hi == l;
    }
  }
};
// Which query tiles may see 128 keys (j0 ... of sequence b).
struct KeyTiles {
  const int32_t* range;  // documents of the query tiles, or null
  int Nq, j0, off, nk, pre, causal, n, lo, hi;
  __device__ __forceinline__ KeyTiles(const AttnArgs& a, int b, int kt, int qtiles, int off_, int nk_, int pre_)
      : Nq(a.Nq), j0(kt * kTile), off(off_), nk(nk_), pre(pre_), causal(a.causal) {
    n = j0 < nk ? qtiles : 0;
    range = a.q_range ? a.q_range + (int64_t)b * qtiles * 2 : nullptr;
    lo = range ? a.k_range[((int64_t)b * a.ktiles + kt) * 2] : 0;
    hi = range ? a.k_range[((int64_t)b * a.ktiles + kt) * 2 + 1] : 0;
  }
  __device__ __forceinline__ int tiles() const { return n; }
  __device__ __forceinline__ void look(int t, bool& see, bool& all) const {
    const int i0 = t * kTile, i1 = min(Nq, i0 + kTile) - 1;
    see = t < n && (!causal || j0 <= max(i1 + off, pre - 1));
    all = j0 + kTile <= nk && (!causal || j0 + kTile - 1 <= max(i0 + off, pre - 1));
    if (see && range) {
      const int32_t l = range[2 * t], h = range[2 * t + 1];
      see = l <= hi && lo <= h;
      all = all && l == h && lo == l && hi == l;
    }
  }
};

// What is said of a step: the first and last of its unit, every row sees the whole tile,
// nothing follows, the tile's columns hold one document.
enum : int32_t { kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8, kOneDoc = 16 };

// Walks the visible tiles in order, 32 at a time by vote: a whole warp calls
// every function together and gets one answer.
template <typename Tiles>
struct TileWalk {
  Tiles v;
  uint32_t see, all;  // the current 32 tiles; visited ones are cleared from `see`
  int word, words;
  __device__ __forceinline__ explicit TileWalk(const Tiles& tiles) : v(tiles), words((tiles.tiles() + 31) >> 5) {
    fetch(0);
  }
  __device__ __forceinline__ void fetch(int w) {
    bool s = false, f = false;
    if (w < words) v.look(w * 32 + (threadIdx.x & 31), s, f);
    word = w;
    see = __ballot_sync(0xffffffffu, s);
    all = __ballot_sync(0xffffffffu, s && f);
  }
  __device__ __forceinline__ int count() const {
    int n = 0;
    for (int w = 0; w < words; ++w) {
      bool s = false, f = false;
      v.look(w * 32 + (threadIdx.x & 31), s, f);
      n += __popc(__ballot_sync(0xffffffffu, s));
    }
    return n;
  }
  // Leaves out the next `rank` tiles.
  __device__ __forceinline__ void skip(int rank) {
    while (word < words) {
      const int n = __popc(see);
      if (rank < n) break;
      rank -= n;
      fetch(word + 1);
    }
    for (; rank > 0; --rank) see &= see - 1;
  }
  // kOneDoc and that document, for a tile given by next()
  __device__ __forceinline__ int one_doc(int j, int& doc) const {
    if (!v.range) return 0;
    doc = v.range[2 * j];
    return doc == v.range[2 * j + 1] ? kOneDoc : 0;
  }
  // The next tile, or -1; `whole`: every row sees all of it.
  __device__ __forceinline__ int next(bool& whole) {
    while (see == 0) {
      if (word + 1 >= words) return -1;
      fetch(word + 1);
    }
    const int bit = __ffs(see) - 1;
    see &= see - 1;
    whole = (all >> bit) & 1;
    return word * 32 + bit;
  }
};

// A CTA's work as the loading warp finds it, one record per step, through a ring in
// shared memory: the other warps need no walk of their own. `tile` is -1 for a unit
// that no tile belongs to (its outputs are still to be written).
struct alignas(16) Record {
  int32_t tile, flags, unit, nk;  // nk, pre: keys_of, prefix_of the unit's sequence
  int32_t pre, doc, b, head;      // doc: with kOneDoc; head: of the unit (key head forward)
  int32_t i0, slot, pad[2];       // first query of the unit; slot of its part, or -1
};
constexpr int kRing = 4;
struct RecordRing {
  Record* slot;     // [kRing]
  uint64_t* full;   // [kRing], one arrival
  uint64_t* empty;  // [kRing], one arrival per reading warp
  volatile int* abort;
  int* err;
  // One thread of the loading warp.
  __device__ __forceinline__ bool put(int r, const Record& rec) const {
    const int s = r % kRing;
    if (r >= kRing && !mbar_wait(&empty[s], (r / kRing - 1) & 1, abort, err)) return false;
    slot[s] = rec;
    mbar_arrive(&full[s]);
    return true;
  }
  __device__ __forceinline__ void end(int r) const {
    Record rec = {};
    rec.tile = -1;
    rec.flags = kEnd;
    put(r, rec);
  }
  // A whole warp: the record's place, or null when the wait gave up. It stays until
  // done(r), so what is needed late is read late.
  __device__ __forceinline__ const Record* at(int r) const {
    return mbar_wait_all(&full[r % kRing], (r / kRing) & 1, abort, err) ? slot + r % kRing : nullptr;
  }
  __device__ __forceinline__ void done(int r) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[r % kRing]);
  }
  // A whole warp: tile and flags, for a warp that needs no more.
  __device__ __forceinline__ int2 get(int r) const {
    const Record* rec = at(r);
    if (!rec) return make_int2(-1, kEnd);
    const int2 v = make_int2(rec->tile, rec->flags);
    done(r);
    return v;
  }
};

// The documents of a step's tile (128 ids), loaded beside its operands where they are read:
// every load is waited for by the warps that compute, so none is under way when a CTA ends. A
// warp that reads record r has finished step r - 1, and record r is written once all have
// read record r - kRing: with twice as many slots a load never meets a reader.
constexpr int kDocRing = 2 * kRing;
// Whether a step with a tile reads the documents of its columns.
__device__ __forceinline__ bool reads_docs(int32_t flags) { return !(flags & (kWhole | kOneDoc)); }
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
struct DocRing {
  int32_t* slot;   // [kDocRing][128]
  uint64_t* full;  // [kDocRing]
  volatile int* abort;
  int* err;
  // The phase of the slot's earlier record has passed (nobody may have waited for it).
  __device__ __forceinline__ bool landed(int r) const {
    return r < kDocRing || mbar_wait(&full[r % kDocRing], (r / kDocRing - 1) & 1, abort, err);
  }
  __device__ __forceinline__ void load(int r, const int32_t* src) const {
    if (!landed(r)) return;
    const int s = r % kDocRing;
    mbar_arrive_expect_tx(&full[s], kTile * 4);
    bulk_load(slot + s * kTile, src, kTile * 4, &full[s]);
  }
  // a record whose documents nobody reads: its slot's phase passes all the same
  __device__ __forceinline__ void skip(int r) const {
    if (landed(r)) mbar_arrive(&full[r % kDocRing]);
  }
  __device__ __forceinline__ const int32_t* get(int r, bool& ok) const {
    const int s = r % kDocRing;
    ok = mbar_wait_all(&full[s], (r / kDocRing) & 1, abort, err);
    return slot + s * kTile;
  }
};

// tanh through one exponential and one reciprocal: absolute error near 2^-22, so the
// capped score is off by 2^-22 of the cap (the one-instruction tanh is off by 2^-11).
__device__ __forceinline__ float tanh_acc(float x) {
  return fmaf(-2.f, fast_rcp(1.f + fast_ex2(2.f * kLog2e * x)), 1.f);
}
// The same, and the slope 1 - tanh^2 = 4 E / (1 + E)^2 with E = e^2x (held below 2^126): right
// to 2^-18 of itself however far x is beyond the cap, where 1 - t t would be rounding.
__device__ __forceinline__ float tanh_slope(float x, float& slope) {
  const float e = fast_ex2(fminf(2.f * kLog2e * x, 126.f)), r = fast_rcp(1.f + e);
  slope = (e * r) * (4.f * r);
  return fmaf(-2.f, r, 1.f);
}

// tanh of two values of magnitude at most 0.75 as x times a polynomial in x^2 (fitted
// for the least relative error, 3e-8): packed FP32 only, where the form above takes
// two operations of the exponential unit, which is what bounds capped scores.
// Capped scores are mostly small beside the cap, so whole rows of a tile take this form.
constexpr float kTanhSmall = 0.75f;
__device__ __forceinline__ void tanh_small2(float x0, float x1, float& t0, float& t1) {
  float y0, y1, p0, p1;
  mul2(x0, x1, x0, x1, y0, y1);
  fma2v(y0, y1, -0.00471625616773963f, -0.00471625616773963f, 0.019582906737923622f, 0.019582906737923622f, p0, p1);
  fma2v(p0, p1, y0, y1, -0.05334442853927612f, -0.05334442853927612f, p0, p1);
  fma2v(p0, p1, y0, y1, 0.1332540661096573f, 0.1332540661096573f, p0, p1);
  fma2v(p0, p1, y0, y1, -0.33332958817481995f, -0.33332958817481995f, p0, p1);
  fma2v(p0, p1, y0, y1, 1.f, 1.f, p0, p1);
  mul2(x0, x1, p0, p1, t0, t1);
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// 32 FP32 values to a row of the output, or of FP32 parts; n of them are inside (a multiple
// of 8). A thread stores a row of its own, so only 32-byte stores fill whole sectors (WIDE:
// where `wide` says that rows start on 32-byte boundaries; 9216 tokens forward: 200 us, 190).
// The kernels with capped or biased scores do without: in an early form of theirs only the
// first element of each such store arrived. The cause was not found, and the present form
// shows nothing of it (forward, with the wide stores put in).
template <bool WIDE, typename T>
__device__ __forceinline__ void store_row32(T* p, const float (&f)[32], int n, bool wide) {
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = Elem<T>::pack(f[i + 2 * j], f[i + 2 * j + 1]);
    if (WIDE && wide && i + 16 <= n) {
      st_global_v8(p + i, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    } else {
      if (i < n) *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
      if (i + 8 < n) *reinterpret_cast<uint4*>(p + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}
// Whether rows of a tensor at p start on 32-byte boundaries.
__device__ __forceinline__ bool wide_rows(const void* p, const int64_t (&s)[3], int D) {
  return D % 16 == 0 && !(reinterpret_cast<uintptr_t>(p) & 31) && !((s[0] | s[1] | s[2]) & 15);
}
__device__ __forceinline__ void store_part32(float* p, const uint32_t (&r)[32], int n) {
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    if (i < n)
      __stcg(reinterpret_cast<float4*>(p + i), make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]),
                                                           __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])));
}

// Ways to cut items (host side).
struct Cut {
  Parts parts;
  int64_t units, slots;
  Cut() {
    memset(this, 0, sizeof(*this));
  }
  void add(int64_t items, int n) {
    if (items <= 0) return;
    const int g = parts.n++;
    parts.item[g] = g ? parts.item[g - 1] + (int32_t)((units - parts.unit[g - 1]) / parts.parts[g - 1]) : 0;
    parts.unit[g] = (int32_t)units;
    parts.parts[g] = n;
    parts.slot[g] = (int32_t)slots;
    units += items * n;
    if (n == 1) return;
    if (!slots) parts.first = parts.item[g];
    parts.count += (int32_t)items;
    slots += items * n;
  }
};
inline Cut cut_even(int64_t items, int n) {
  Cut c;
  c.add(items, n);
  return c;
}
// the last `rest` items
inline Cut cut_last(int64_t items, int64_t rest, int n) {
  Cut c;
  c.add(items - rest, 1);
  c.add(rest, n);
  return c;
}
// Items whose lengths fall evenly from `longest` to `least`: parts of at most 1 / k of the
// longest (k <= kGroups).
inline Cut cut_levels(int64_t items, int k, double longest, double least) {
  Cut c;
  int64_t done = 0;
  for (int n = k; n >= 1; --n) {
    const double to = longest > least ? (longest - longest * (n - 1) / k) / (longest - least) : 1.0;
    const int64_t end = n == 1 ? items : (int64_t)(items * (to < 1.0 ? to : 1.0));
    if (end > done) c.add(end - done, n);
    done = end > done ? end : done;
  }
  return c;
}

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
// The backward pass (attention_grad.cu).
size_t attn_grad_space(const sd_attention_cfg& c);
template <typename T>
sd_status attn_backward(AttnCall& c);
// Map of a [batch][tokens][heads][D] tensor; a box holds box_heads x box_tokens rows of 64.
bool attn_map(CUtensorMap* m, bool f16, const void* p, const int64_t* s, int batch, int tokens, int heads, int d,
              uint32_t box_heads, uint32_t box_tokens);
// Lowest and highest document id of each key tile and of each tile of `tq` queries, and
// the ids in rows of whole tiles.
sd_status attn_doc_ranges(const AttnArgs& a, int tq, cudaStream_t st);
void attn_fill(AttnCall& c, const sd_attention_masks* m);

}  // namespace sdo
