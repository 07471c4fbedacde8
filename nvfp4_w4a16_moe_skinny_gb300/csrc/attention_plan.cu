// The split of an attention call, walked on the host through the kernels' own arithmetic
// (paged_attention_plan_check): which range of units holds which share of which item, where the
// shares go, and how the joins of the tcgen05 kernel's split items come out under different
// orders of arrival.  (The kernels find a range's first item by a scan over the sequences,
// find_range; here the items are numbered one after the other.)
#include <algorithm>
#include <new>
#include <vector>

#include "attention_chunk.cuh"

namespace nvfp4 {
namespace {

template <int kDim, bool kFp8>
Tiling tiling_at(const AttnShape& s) {
  if (s.chunk) return ChunkTile<kDim, kFp8>::tiling();
  if (s.rw == 1) return AttnTile<kDim, kFp8, 1, 4>::tiling();
  if (s.rw == 2) return AttnTile<kDim, kFp8, 2, 2>::tiling();
  return AttnTile<kDim, kFp8, 4, 1>::tiling();
}

Tiling tiling_of(int dim, bool fp8, const AttnShape& s) {
  if (dim == 64) return fp8 ? tiling_at<64, true>(s) : tiling_at<64, false>(s);
  if (dim == 128) return fp8 ? tiling_at<128, true>(s) : tiling_at<128, false>(s);
  return fp8 ? tiling_at<256, true>(s) : tiling_at<256, false>(s);
}

struct Split {
  int c0, holders;
};
struct Held {  // a CTA's share of a split item: which one, and its place among the item's
  int item, mine;
};

// The join of the tcgen05 kernel's split items, one step of one CTA at a time in some order:
// the items that are not joined exactly once, from all their shares, and the counters left
// behind.  `held` lists every CTA's shares in the order in which it comes to them.
struct Arrivals {
  const std::vector<Split>& items;
  const std::vector<std::vector<Held>>& held;

  // order 0: the CTAs one after the other, 1: from the last to the first, else at random
  long long wrong(int order) const {
    const int ctas = static_cast<int>(held.size());
    std::vector<unsigned> counter(kAttnCounterBytes / sizeof(unsigned) / 2, 0);
    std::vector<std::vector<int>> parts(items.size());  // holders' shares that each share stands for, 0 before it is written
    for (size_t i = 0; i < items.size(); ++i) parts[i].assign(items[i].holders, 0);
    std::vector<int> joined(items.size(), 0), at(ctas, 0), level(ctas, 0), mine(ctas, -1);
    std::vector<int> active;
    for (int c = 0; c < ctas; ++c)
      if (!held[c].empty()) active.push_back(c);
    long long bad = 0;
    uint64_t state = 0x9E3779B97F4A7C15ull * (order + 1);
    while (!active.empty()) {
      state = state * 6364136223846793005ull + 1442695040888963407ull;
      const size_t pick = order == 0 ? 0 : (order == 1 ? active.size() - 1 : (state >> 33) % active.size());
      const int c = active[pick];
      const Held h = held[c][at[c]];
      const Split& it = items[h.item];
      if (mine[c] < 0) mine[c] = h.mine, level[c] = 0, parts[h.item][h.mine] = 1;
      const JoinStep s = join_step(mine[c], level[c], it.holders);
      bool next = true;  // on to the CTA's next share
      if (s.counter >= 0) {
        unsigned& n = counter[it.c0 + s.counter];
        const bool last = n++ == static_cast<unsigned>(s.count - 1);
        if (last) {
          n = 0;
          int all = 0;
          for (int i = 0; i < s.count; ++i) {
            const int share = s.start + i * s.stride;
            if (parts[h.item][share] != std::min(s.stride, it.holders - share)) ++bad;  // joined too early
            all += parts[h.item][share];
          }
          parts[h.item][s.start] = all;
          if (s.top)
            ++joined[h.item];
          else
            next = false;
        }
      } else {
        next = false;
      }
      if (next) {
        mine[c] = -1;
        if (++at[c] == static_cast<int>(held[c].size())) active.erase(active.begin() + pick);
      } else {
        mine[c] = s.start;
        ++level[c];
      }
    }
    for (int j : joined) bad += j != 1;
    for (unsigned n : counter) bad += n != 0;
    return bad;
  }
};

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

static nvfp4_status plan_check(const nvfp4_kv_cache* cache, const nvfp4_batch* batch, int32_t n_tokens, int32_t n_heads,
                               int32_t window, int32_t orders, int32_t* out, int32_t out_len) {
  if (const nvfp4_status st = check_cache(cache)) return st;
  if (!batch || !out || !batch->cu_tokens || !batch->kv_len) return NVFP4_ERR_NULL;
  const int kv = cache->n_kv_heads, dim = cache->head_dim;
  if (out_len < 9 || orders < 0 || window < 0) return NVFP4_ERR_SHAPE;
  if (!attn_sizes_ok(n_tokens, batch->n_seqs, batch->max_new, n_heads, kv, dim, batch->max_pages, cache->page_size))
    return NVFP4_ERR_SHAPE;
  const bool fp8 = cache->dtype == NVFP4_KV_E4M3;
  const AttnShape shape = attn_shape(dim, fp8, packed_rows(n_tokens, batch->max_new, n_heads, kv),
                                     static_cast<int64_t>(batch->n_seqs) * kv);
  const Tiling g = tiling_of(dim, fp8, shape);
  const int ctas = kAttnGrid * (shape.chunk ? 1 : attn_ctas(dim, fp8, shape.rw));
  AttnJob p{};
  p.n_seqs = batch->n_seqs, p.max_pages = batch->max_pages, p.n_tokens = n_tokens;
  p.n_heads = n_heads, p.n_kv = kv, p.group = n_heads / kv, p.by_group = fast_div(n_heads / kv);
  p.page_log2 = log2i(cache->page_size), p.window = attn_window(window);

  const auto each_tile = [&](auto f) {
    for (int b = 0; b < p.n_seqs; ++b) {
      Walk w{};
      w.b = b;
      w.s = sequence_from(p, batch->cu_tokens[b], batch->cu_tokens[b + 1], batch->kv_len[b], g);
      for (w.rt = 0; w.rt < w.s.tiles; ++w.rt) {
        w.t = row_tile(p, w.s, w.rt, g);
        f(w);
      }
    }
  };
  long long total = 0, n_items = 0;
  each_tile([&](const Walk& w) { total += static_cast<long long>(w.t.units + g.over) * kv, n_items += kv; });
  if (n_items > (1 << 22)) return NVFP4_ERR_SHAPE;
  Ranges r{};
  r.set(total, ctas, g.least);

  long long bad = 0, shared = 0, unjoined = 0;
  int most = 0;
  std::vector<Split> items;
  std::vector<std::vector<Held>> held(ctas);
  std::vector<uint8_t> slots(2 * ctas, 0), starts(ctas, 0);
  if (r.grid > 0 && (r.start(0) != 0 || r.start(r.grid) != total)) ++bad;
  long long at = 0;
  each_tile([&](Walk w) {
    const int span = w.t.units + g.over;
    for (w.h = 0; w.h < kv; ++w.h, at += span) {
      w.item0 = at;
      const Holders h = holders_of(w, r, g);
      int tile = w.t.tile0, holders = 0;
      for (int c = r.holder(at); c <= r.holder(at + span - 1); ++c) {
        const long long u0 = r.start(c), u1 = r.start(c + 1);
        const Share q = share_at(w, std::max(at, u0), u0, u1, c, g);
        if (q.end != std::min(at + span, u1)) ++bad;
        if (q.n == 0) continue;
        if (q.first != tile) ++bad;  // the item's tiles one after the other, each once
        tile += q.n;
        if (q.whole) {
          if (h.c0 != h.c1) ++bad;
          continue;
        }
        // the place where the join looks for it
        if (c != h.c0 + holders || q.slot != 2 * c + (c == h.c0)) ++bad;
        if (q.slot < 0 || q.slot >= 2 * ctas || slots[q.slot]++) ++bad;
        held[c].push_back({static_cast<int>(items.size()), holders++});
      }
      if (tile != w.t.tile0 + w.t.units) ++bad;
      if (holders == 0) continue;
      if (h.c0 + holders - 1 != h.c1 || holders < 2 || starts[h.c0]++) ++bad;  // (one split item starts in a range)
      most = std::max(most, holders);
      items.push_back({h.c0, holders});
    }
  });
  if (shape.chunk && bad == 0) {
    std::vector<int> owner(kAttnCounterBytes / sizeof(unsigned) / 2, -1);
    for (size_t i = 0; i < items.size(); ++i)
      for (int m = 0; m < items[i].holders; ++m)
        for (int level = 0;; ++level) {
          const JoinStep s = join_step(m, level, items[i].holders);
          if (s.counter >= 0) {
            const int n = items[i].c0 + s.counter;
            if (n >= static_cast<int>(owner.size())) return NVFP4_ERR_SHAPE;  // past the workspace's counters
            if (owner[n] >= 0 && owner[n] != static_cast<int>(i)) ++shared;
            owner[n] = static_cast<int>(i);
          }
          if (s.top) break;
        }
    for (int o = 0; o < orders; ++o) unjoined += Arrivals{items, held}.wrong(o);
  }
  const auto fits = [](long long v) { return static_cast<int32_t>(std::min<long long>(v, 0x7fffffff)); };
  out[0] = bad == 0 && shared == 0 && unjoined == 0;
  out[1] = g.rows;
  out[2] = r.grid;
  out[3] = fits(n_items);
  out[4] = fits(static_cast<long long>(items.size()));
  out[5] = most;
  out[6] = fits(shared);
  out[7] = fits(unjoined);
  out[8] = shape.chunk ? 1 : 0;
  return NVFP4_OK;
}

extern "C" nvfp4_status paged_attention_plan_check(const nvfp4_kv_cache* cache, const nvfp4_batch* batch,
                                                   int32_t n_tokens, int32_t n_heads, int32_t window, int32_t orders,
                                                   int32_t* out, int32_t out_len) {
  try {
    return plan_check(cache, batch, n_tokens, n_heads, window, orders, out, out_len);
  } catch (const std::bad_alloc&) {  // (nothing else is thrown)
    return NVFP4_ERR_WORKSPACE;
  }
}
