// The tree kernels' list (csrc/tree_list.cuh) under a scheduler of its own: the roles are threads of which one runs at a
// time, chosen at random wherever another one's step could matter.  Waits run out at random, and roles run out of
// other waits between items.  Prints "ok", or what went wrong: an item that changed while it was read, one that is
// not the next, roles that never end.
//   tree_list SEEDS
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "tree_list.cuh"

namespace {

struct Run {
  std::mutex mu;
  std::condition_variable cv;
  int turn = -1;  // the role that runs
  std::vector<bool> ended;
  uint64_t state;
  long steps = 0;
  std::string wrong;

  uint32_t random(uint32_t n) {  // (a linear congruential generator's high half)
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return static_cast<uint32_t>(state >> 33) % n;
  }
  void next() {  // with the lock held
    ++steps;
    std::vector<int> left;
    for (size_t i = 0; i < ended.size(); ++i)
      if (!ended[i]) left.push_back(static_cast<int>(i));
    turn = left.empty() ? -1 : left[random(static_cast<uint32_t>(left.size()))];
    cv.notify_all();
  }
  void pass(int me) {
    std::unique_lock<std::mutex> lock(mu);
    next();
    cv.wait(lock, [&] { return turn == me; });
  }
  void fail(const std::string& what) {
    if (wrong.empty()) wrong = what;
  }
};

struct Barrier {
  int count, pending;
  uint32_t phase = 0;  // completed so far
  void arrive() {
    if (--pending == 0) ++phase, pending = count;
  }
};

Run* run;
thread_local int me;
std::map<const uint64_t*, Barrier> barriers;

// An item whose copies can be watched half done.
struct Item {
  int n = 0, id[3] = {-1, -1, -1};
  Item() = default;
  Item(int tiles, int i) : n(tiles), id{i, i, i} {}
  Item(const Item& o) { *this = o; }
  Item& operator=(const Item& o) {
    n = o.n;
    for (int k = 0; k < 3; ++k) {
      id[k] = o.id[k];
      run->pass(me);
    }
    return *this;
  }
};

struct By {
  int patience;  // turns that a wait lasts
  bool wait(const uint64_t* bar, uint32_t parity) const {
    for (int i = 0; i < patience; ++i) {
      // the phase that ends with this parity is complete
      if ((barriers.at(bar).phase & 1) != parity) return true;
      run->pass(me);
    }
    return false;
  }
  void leave(uint64_t* bar) const {
    run->pass(me);
    barriers.at(bar).arrive();
  }
  template <typename Fill>
  void put(Item& slot, const Fill& fill, uint64_t* full) const {
    fill(slot);
    barriers.at(full).arrive();
  }
};

std::string one(uint64_t seed) {
  Run r;
  run = &r;
  r.state = seed * 0x9E3779B97F4A7C15ull + 1;
  nvfp4::ItemList<Item> list;
  const int readers = 2 + static_cast<int>(r.random(5)), items = static_cast<int>(r.random(14));
  const bool calm = r.random(4) == 0;  // nobody runs out of anything
  const int patience = calm ? 1 << 30 : 20 + static_cast<int>(r.random(400)), quits = calm ? 0 : static_cast<int>(r.random(3));
  std::vector<int> quit_at(readers + 1, 1 << 30), read(readers, 0);
  for (int i = 0; i < quits; ++i) quit_at[r.random(readers + 1)] = static_cast<int>(r.random(items + 1));
  barriers.clear();
  for (int i = 0; i < list.kSlots; ++i) {
    barriers[list.full + i] = Barrier{1, 1};
    barriers[list.empty + i] = Barrier{readers, readers};
  }
  r.ended.assign(readers + 1, false);
  bool all_put = false;
  const auto role = [&](int who) {
    me = who;
    {
      std::unique_lock<std::mutex> lock(r.mu);
      r.cv.wait(lock, [&] { return r.turn == who; });
    }
    const By by{patience};
    bool ran_out = false;
    if (who == readers) {  // the writer
      int at = 0;
      for (int i = 0; i < items && !ran_out; ++i) {
        at += nvfp4::put_item(list, at, [&](Item& slot) { slot = Item(1 + i % 3, i); }, by, ran_out);
        ran_out = ran_out || i == quit_at[who];
      }
      all_put = nvfp4::put_item(list, at, [&](Item& slot) { slot = Item(0, at); }, by, ran_out) && at == items;
    } else {
      const bool looks = who % 2 == 0;
      for (int i = 0;; ++i) {
        Item x;
        if (!nvfp4::take_item(list, i, [&](const Item& slot) { x = slot; }, by, ran_out)) break;
        if (x.id[0] != i || x.id[1] != i || x.id[2] != i) r.fail("an item that is not the next, or half of it");
        if (x.n == 0) break;
        ++read[who];
        r.pass(me);  // work
        ran_out = ran_out || i == quit_at[who];
        if (looks) {
          Item ahead;
          if (nvfp4::look_at_item(list, i + 1, [&](const Item& slot) { ahead = slot; }, by, ran_out) && (ahead.id[0] != i + 1 || ahead.id[2] != i + 1))
            r.fail("an item ahead that is not the next, or half of it");
        }
      }
    }
    std::unique_lock<std::mutex> lock(r.mu);
    r.ended[who] = true;
    r.next();
  };
  std::vector<std::thread> threads;
  for (int i = 0; i <= readers; ++i) threads.emplace_back(role, i);
  {
    std::unique_lock<std::mutex> lock(r.mu);
    r.next();
  }
  for (auto& t : threads) t.join();
  if (calm) {
    if (!all_put) r.fail("items left out although no wait ran out");
    for (int n : read)
      if (n != items) r.fail("a reader without all items although no wait ran out");
  }
  return r.wrong;
}

}  // namespace

int main(int argc, char** argv) {
  const int seeds = argc > 1 ? std::atoi(argv[1]) : 100;
  for (int i = 0; i < seeds; ++i) {
    const std::string wrong = one(i);
    if (!wrong.empty()) {
      std::printf("seed %d: %s\n", i, wrong.c_str());
      return 1;
    }
  }
  std::printf("ok\n");
}
