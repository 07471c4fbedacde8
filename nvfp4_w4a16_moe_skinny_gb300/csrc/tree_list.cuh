// The list of items that the roles of a tree kernel's CTA work through: one warp finds them and
// puts them in, the others read them, all of them in order.  Plain C++ but for the waits and arrivals, which the
// caller brings, so that the host can walk it too.
//
// Every wait has a limit.  A role that has run out of one (`ran_out`) leaves the list: what it finds in a slot,
// which may be written meanwhile, is not used, and it does not say that it has read it, as its arrival would then
// stand for another reader's.  The writer fills a slot only after all readers have said so.  So a slot holds still
// while it is used, whoever has left, and the ones that stay run out of their own waits in turn.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define NVFP4_BOTH __host__ __device__ __forceinline__
#else
#define NVFP4_BOTH inline
#endif

namespace nvfp4 {

template <typename Item>
struct ItemList {
  static constexpr int kSlots = 4;
  uint64_t full[kSlots], empty[kSlots];  // barriers: the writer's arrival; one of each reader
  Item item[kSlots];
};

// Item i from the writer, by fill(slot): false, with nothing written, if its slot's readers do not come in time.
template <typename Item, typename Fill, typename By>
NVFP4_BOTH bool put_item(ItemList<Item>& list, int i, const Fill& fill, const By& by, bool& ran_out) {
  constexpr int kSlots = ItemList<Item>::kSlots;
  // (whatever else ran out, the slot is not the writer's before they have: a wait of its own)
  if (i >= kSlots && !by.wait(list.empty + i % kSlots, (i / kSlots - 1) & 1)) {
    ran_out = true;
    return false;
  }
  by.put(list.item[i % kSlots], fill, list.full + i % kSlots);
  return true;
}

// Item i to a reader, by read(slot), who keeps the slot: false, with nothing of use read, if it has run out of a wait,
// this one or an earlier one.  (Read all the same, not past a branch: that cost the kernels registers.)
template <typename Item, typename Read, typename By>
NVFP4_BOTH bool look_at_item(const ItemList<Item>& list, int i, const Read& read, const By& by, bool& ran_out) {
  constexpr int kSlots = ItemList<Item>::kSlots;
  ran_out = ran_out || !by.wait(list.full + i % kSlots, i / kSlots & 1);
  read(list.item[i % kSlots]);
  return !ran_out;
}

// The same, and the slot goes back to the writer.
template <typename Item, typename Read, typename By>
NVFP4_BOTH bool take_item(ItemList<Item>& list, int i, const Read& read, const By& by, bool& ran_out) {
  const bool came = look_at_item(list, i, read, by, ran_out);
  if (came) by.leave(list.empty + i % ItemList<Item>::kSlots);
  return came;
}

}  // namespace nvfp4
