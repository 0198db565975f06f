// Host PageTable allocator with an optional device mirror of the table.
//
// Policy from "unsloth: compare main...transformers-continuous-batching-qwen3"
// · scripts/benchmarks/flex_paged_attention.py · class PageTable, with the
// +1 capacity rule from the commit message on "unsloth: compare
// main...flex-moe-qwen3":
//   - slot 0 is a no-op slot whose table row is all page 0; page 0 is a dummy
//     page; user max_batch_size N -> N usable slots 1..N (N+1 rows);
//   - free slots and free pages are LIFO stacks, initially [N..1] and
//     [n_pages-1..1] (the back of each vector is the top);
//   - allocate pops a slot, zeroes its capacity and resets its row to -1;
//   - reserve takes the last k free pages in list order for the next k
//     logical blocks, or fails with no change;
//   - erase pushes the slot and appends its pages in reverse order; the
//     device row stays stale until the slot is allocated again.
// Pages may be shared by several slots (pt_fork): each page counts the slots
// that hold it and returns to the free stack when the last one lets go.
// The host keeps the authoritative copy so no call reads device memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <new>
#include <vector>

#include "pkv_internal.h"

struct pkv_pt {
  int max_batch_size = 0;
  int n_slots = 0;
  int page_size = 0;
  int n_pages = 0;
  int max_pages = 0;
  int32_t *dev_table = nullptr;
  cudaStream_t stream = nullptr;
  std::vector<int32_t> table;              // [n_slots][max_pages]
  std::vector<int> capacity;               // tokens per slot
  std::vector<std::vector<int32_t>> pages; // pages per slot, logical order
  std::vector<int32_t> refs;               // slots holding each page (0: free)
  std::vector<int32_t> free_pages;         // back = next taken
  std::vector<int> free_slots;             // back = next popped
  std::vector<char> live;                  // slot allocated?
};

namespace {

int pages_needed(int cap, int seq_len, int ps) {
  if (seq_len <= cap) return 0;
  return static_cast<int>((static_cast<long long>(seq_len) - cap + ps - 1) / ps);
}

// Whether a slot of `cap` tokens may have k more pages: the row has room and the capacity
// stays within an int.
bool row_holds(const pkv_pt *pt, int cap, int k) {
  return static_cast<long long>(cap) / pt->page_size + k <= pt->max_pages &&
         cap + static_cast<long long>(k) * pt->page_size <= 0x7fffffffLL;
}

int write_row_range(pkv_pt *pt, int slot, int begin, long long count) {
  if (!pt->dev_table || count <= 0) return PKV_OK;
  size_t off = static_cast<size_t>(slot) * pt->max_pages + begin;
  PKV_CUDA_CHECK(cudaMemcpyAsync(pt->dev_table + off, pt->table.data() + off,
                                 sizeof(int32_t) * count,
                                 cudaMemcpyHostToDevice, pt->stream));
  return PKV_OK;
}

// Lets go of one hold on page p.
void release_page(pkv_pt *pt, int32_t p) {
  if (--pt->refs[p] == 0) pt->free_pages.push_back(p);
}

bool valid_live(const pkv_pt *pt, int slot) {
  return slot >= 1 && slot < pt->n_slots && pt->live[slot];
}

}  // namespace

extern "C" {

int pt_create(int max_batch_size, int page_size, int n_pages,
              int max_pages_per_seq, int32_t *dev_table, void *stream,
              pkv_pt **out) {
  if (!out) return pkv::fail(PKV_E_BAD_ARG, "pt_create: out is NULL");
  if (max_batch_size < 1 || max_batch_size == 0x7fffffff || page_size < 1 || n_pages < 2 ||
      max_pages_per_seq < 1)
    return pkv::fail(PKV_E_BAD_ARG,
                     "pt_create: need max_batch_size>=1, page_size>=1, "
                     "n_pages>=2, max_pages_per_seq>=1");
  if (dev_table && (reinterpret_cast<uintptr_t>(dev_table) & 3u))
    return pkv::fail(PKV_E_BAD_ARG, "pt_create: dev_table not 4-byte aligned");
  pkv_pt *pt = new (std::nothrow) pkv_pt();
  if (!pt) return pkv::fail(PKV_E_BAD_ARG, "pt_create: out of host memory");
  pt->max_batch_size = max_batch_size;
  pt->n_slots = max_batch_size + 1;
  pt->page_size = page_size;
  pt->n_pages = n_pages;
  pt->max_pages = max_pages_per_seq;
  pt->dev_table = dev_table;
  pt->stream = static_cast<cudaStream_t>(stream);
  try {
    pt->table.assign(static_cast<size_t>(pt->n_slots) * max_pages_per_seq, -1);
    std::fill(pt->table.begin(), pt->table.begin() + max_pages_per_seq, 0);
    pt->capacity.assign(pt->n_slots, 0);
    pt->pages.assign(pt->n_slots, {});
    pt->live.assign(pt->n_slots, 0);
    pt->refs.assign(n_pages, 0);
    pt->free_pages.reserve(n_pages);
    for (int p = n_pages - 1; p >= 1; --p) pt->free_pages.push_back(p);
    for (int s = max_batch_size; s >= 1; --s) pt->free_slots.push_back(s);
  } catch (...) {
    delete pt;
    return pkv::fail(PKV_E_BAD_ARG, "pt_create: out of host memory");
  }
  int st = write_row_range(pt, 0, 0, 1LL * pt->n_slots * max_pages_per_seq);
  if (st != PKV_OK) {
    delete pt;
    return st;
  }
  *out = pt;
  return pkv::ok();
}

int pt_destroy(pkv_pt *pt) {
  delete pt;
  return pkv::ok();
}

int pt_set_stream(pkv_pt *pt, void *stream) {
  if (!pt) return pkv::fail(PKV_E_BAD_ARG, "pt_set_stream: NULL handle");
  pt->stream = static_cast<cudaStream_t>(stream);
  return pkv::ok();
}

int pt_get_stream(const pkv_pt *pt, void **stream) {
  if (!pt || !stream) return pkv::fail(PKV_E_BAD_ARG, "pt_get_stream: NULL");
  *stream = pt->stream;
  return pkv::ok();
}

int pt_can_reserve(const pkv_pt *pt, int seq_len, int slot, int *ok) {
  if (!pt || !ok) return pkv::fail(PKV_E_BAD_ARG, "pt_can_reserve: NULL");
  if (slot < 0) {
    int k = pages_needed(0, seq_len, pt->page_size);
    *ok = !pt->free_slots.empty() &&
          static_cast<long long>(pt->free_pages.size()) * pt->page_size >=
              seq_len &&
          row_holds(pt, 0, k);
    return pkv::ok();
  }
  if (!valid_live(pt, slot))
    return pkv::fail(PKV_E_BAD_SLOT, "pt_can_reserve: slot %d not allocated",
                     slot);
  int cap = pt->capacity[slot];
  int k = pages_needed(cap, seq_len, pt->page_size);
  *ok = k <= static_cast<int>(pt->free_pages.size()) && row_holds(pt, cap, k);
  return pkv::ok();
}

static int reserve_impl(pkv_pt *pt, int slot, int seq_len) {
  int cap = pt->capacity[slot];
  int k = pages_needed(cap, seq_len, pt->page_size);
  if (k == 0) return PKV_OK;
  int start = cap / pt->page_size;
  if (!row_holds(pt, cap, k))
    return pkv::fail(PKV_E_BAD_ARG,
                     "reserve: %d tokens exceed the table row (%d pages)",
                     seq_len, pt->max_pages);
  if (k > static_cast<int>(pt->free_pages.size()))
    return pkv::fail(PKV_E_NO_PAGES, "reserve: need %d pages, %zu free", k,
                     pt->free_pages.size());
  try {
    pt->pages[slot].reserve(pt->pages[slot].size() + k);
  } catch (...) {
    return pkv::fail(PKV_E_BAD_ARG, "reserve: out of host memory");
  }
  // take the tail free_pages[-k:] in list order for blocks start..start+k-1
  size_t first = pt->free_pages.size() - k;
  int32_t *row = pt->table.data() + static_cast<size_t>(slot) * pt->max_pages;
  for (int i = 0; i < k; ++i) {
    int32_t p = pt->free_pages[first + i];
    row[start + i] = p;
    pt->pages[slot].push_back(p);
    pt->refs[p] = 1;
  }
  pt->free_pages.resize(first);
  pt->capacity[slot] = cap + k * pt->page_size;
  return PKV_OK;
}

int pt_reserve(pkv_pt *pt, int slot, int seq_len) {
  if (!pt) return pkv::fail(PKV_E_BAD_ARG, "pt_reserve: NULL handle");
  if (!valid_live(pt, slot))
    return pkv::fail(PKV_E_BAD_SLOT, "pt_reserve: slot %d not allocated", slot);
  if (seq_len < 0) return pkv::fail(PKV_E_BAD_ARG, "pt_reserve: negative length");
  int start = pt->capacity[slot] / pt->page_size;
  size_t before = pt->pages[slot].size();
  int st = reserve_impl(pt, slot, seq_len);
  if (st != PKV_OK) return st;
  int added = static_cast<int>(pt->pages[slot].size() - before);
  st = write_row_range(pt, slot, start, added);
  if (st != PKV_OK) return st;
  return pkv::ok();
}

int pt_assign(pkv_pt *pt, int seq_len, int *slot_out) {
  if (!pt || !slot_out) return pkv::fail(PKV_E_BAD_ARG, "pt_assign: NULL");
  if (seq_len < 0) return pkv::fail(PKV_E_BAD_ARG, "pt_assign: negative length");
  if (pt->free_slots.empty())
    return pkv::fail(PKV_E_NO_SLOT, "pt_assign: no free slot");
  int k = pages_needed(0, seq_len, pt->page_size);
  if (!row_holds(pt, 0, k))
    return pkv::fail(PKV_E_BAD_ARG,
                     "pt_assign: %d tokens exceed the table row (%d pages)",
                     seq_len, pt->max_pages);
  if (k > static_cast<int>(pt->free_pages.size()))
    return pkv::fail(PKV_E_NO_PAGES, "pt_assign: need %d pages, %zu free", k,
                     pt->free_pages.size());
  int slot = pt->free_slots.back();
  try {   // room first, so that nothing below can fail
    pt->pages[slot].reserve(k);
  } catch (...) {
    return pkv::fail(PKV_E_BAD_ARG, "pt_assign: out of host memory");
  }
  pt->free_slots.pop_back();
  pt->live[slot] = 1;
  pt->capacity[slot] = 0;
  pt->pages[slot].clear();
  int32_t *row = pt->table.data() + static_cast<size_t>(slot) * pt->max_pages;
  std::fill(row, row + pt->max_pages, -1);
  int st = reserve_impl(pt, slot, seq_len);  // cannot fail after the checks
  if (st == PKV_OK) st = write_row_range(pt, slot, 0, pt->max_pages);
  if (st != PKV_OK) return st;
  *slot_out = slot;
  return pkv::ok();
}

int pt_free(pkv_pt *pt, int slot) {
  if (!pt) return pkv::fail(PKV_E_BAD_ARG, "pt_free: NULL handle");
  if (!valid_live(pt, slot))
    return pkv::fail(PKV_E_BAD_SLOT, "pt_free: slot %d not allocated", slot);
  pt->free_slots.push_back(slot);
  pt->live[slot] = 0;
  auto &pg = pt->pages[slot];
  for (auto it = pg.rbegin(); it != pg.rend(); ++it) release_page(pt, *it);
  pg.clear();
  pt->capacity[slot] = 0;
  return pkv::ok();
}

// The new slots share the pages that seq_len tokens fill; each gets a page of
// its own for the partly filled last one, which the caller copies (pairs).
int pt_fork(pkv_pt *pt, int src_slot, int seq_len, int count, int *slots_out,
            int32_t *pairs_out, int max_pairs, int *n_pairs) {
  if (!pt || !slots_out || !n_pairs) return pkv::fail(PKV_E_BAD_ARG, "pt_fork: NULL");
  if (!valid_live(pt, src_slot))
    return pkv::fail(PKV_E_BAD_SLOT, "pt_fork: slot %d not allocated", src_slot);
  if (count < 1) return pkv::fail(PKV_E_BAD_ARG, "pt_fork: count must be >= 1");
  if (seq_len < 0 || seq_len > pt->capacity[src_slot])
    return pkv::fail(PKV_E_BAD_ARG, "pt_fork: %d tokens, slot %d holds %d", seq_len, src_slot,
                     pt->capacity[src_slot]);
  if (count > static_cast<int>(pt->free_slots.size()))
    return pkv::fail(PKV_E_NO_SLOT, "pt_fork: need %d slots, %zu free", count,
                     pt->free_slots.size());
  const int shared = seq_len / pt->page_size;
  const bool tail = seq_len % pt->page_size != 0;
  const int need = tail ? count : 0;
  if (need > static_cast<int>(pt->free_pages.size()))
    return pkv::fail(PKV_E_NO_PAGES, "pt_fork: need %d pages, %zu free", need,
                     pt->free_pages.size());
  if (need > 0 && (!pairs_out || max_pairs < need))
    return pkv::fail(PKV_E_BAD_ARG, "pt_fork: room for %d pairs needed", need);
  try {   // room first, so that nothing below can throw
    for (int i = 0; i < count; ++i)
      pt->pages[pt->free_slots[pt->free_slots.size() - 1 - i]].reserve(shared + 1);
  } catch (...) {
    return pkv::fail(PKV_E_BAD_ARG, "pt_fork: out of host memory");
  }
  const int32_t *from = pt->table.data() + static_cast<size_t>(src_slot) * pt->max_pages;
  for (int i = 0; i < count; ++i) {
    const int slot = pt->free_slots.back();
    pt->free_slots.pop_back();
    pt->live[slot] = 1;
    int32_t *row = pt->table.data() + static_cast<size_t>(slot) * pt->max_pages;
    std::fill(row, row + pt->max_pages, -1);
    pt->pages[slot].clear();
    for (int b = 0; b < shared; ++b) {
      row[b] = from[b];
      pt->pages[slot].push_back(from[b]);
      ++pt->refs[from[b]];
    }
    if (tail) {
      const int32_t p = pt->free_pages.back();
      pt->free_pages.pop_back();
      pt->refs[p] = 1;
      row[shared] = p;
      pt->pages[slot].push_back(p);
      pairs_out[2 * i] = from[shared];
      pairs_out[2 * i + 1] = p;
    }
    pt->capacity[slot] = static_cast<int>(pt->pages[slot].size()) * pt->page_size;
    slots_out[i] = slot;
  }
  *n_pairs = need;
  for (int i = 0; i < count; ++i) {
    const int st = write_row_range(pt, slots_out[i], 0, pt->max_pages);
    if (st != PKV_OK) return st;
  }
  return pkv::ok();
}

// Gives the slot pages of its own for the shared ones under tokens [begin, end).
int pt_unshare(pkv_pt *pt, int slot, int begin, int end, int32_t *pairs_out, int max_pairs,
               int *n_pairs) {
  if (!pt || !n_pairs) return pkv::fail(PKV_E_BAD_ARG, "pt_unshare: NULL");
  if (!valid_live(pt, slot))
    return pkv::fail(PKV_E_BAD_SLOT, "pt_unshare: slot %d not allocated", slot);
  if (begin < 0 || end < begin || end > pt->capacity[slot])
    return pkv::fail(PKV_E_BAD_ARG, "pt_unshare: tokens [%d, %d), slot %d holds %d", begin, end,
                     slot, pt->capacity[slot]);
  const int b0 = begin / pt->page_size;
  const int b1 = end > begin ? (end - 1) / pt->page_size + 1 : b0;
  int need = 0;
  for (int b = b0; b < b1; ++b) need += pt->refs[pt->pages[slot][b]] > 1;
  if (need > static_cast<int>(pt->free_pages.size()))
    return pkv::fail(PKV_E_NO_PAGES, "pt_unshare: need %d pages, %zu free", need,
                     pt->free_pages.size());
  if (need > 0 && (!pairs_out || max_pairs < need))
    return pkv::fail(PKV_E_BAD_ARG, "pt_unshare: room for %d pairs needed", need);
  int32_t *row = pt->table.data() + static_cast<size_t>(slot) * pt->max_pages;
  int n = 0;
  for (int b = b0; b < b1; ++b) {
    const int32_t old = pt->pages[slot][b];
    if (pt->refs[old] <= 1) continue;
    const int32_t p = pt->free_pages.back();
    pt->free_pages.pop_back();
    pt->refs[p] = 1;
    --pt->refs[old];
    pt->pages[slot][b] = row[b] = p;
    pairs_out[2 * n] = old;
    pairs_out[2 * n + 1] = p;
    ++n;
  }
  *n_pairs = n;
  if (n > 0) {
    const int st = write_row_range(pt, slot, b0, b1 - b0);
    if (st != PKV_OK) return st;
  }
  return pkv::ok();
}

int pt_truncate(pkv_pt *pt, int slot, int seq_len) {
  if (!pt) return pkv::fail(PKV_E_BAD_ARG, "pt_truncate: NULL handle");
  if (!valid_live(pt, slot))
    return pkv::fail(PKV_E_BAD_SLOT, "pt_truncate: slot %d not allocated", slot);
  if (seq_len < 0 || seq_len > pt->capacity[slot])
    return pkv::fail(PKV_E_BAD_ARG, "pt_truncate: %d tokens, slot %d holds %d", seq_len, slot,
                     pt->capacity[slot]);
  const int keep = pages_needed(0, seq_len, pt->page_size);
  auto &pg = pt->pages[slot];
  const int had = static_cast<int>(pg.size());
  if (keep == had) return pkv::ok();
  int32_t *row = pt->table.data() + static_cast<size_t>(slot) * pt->max_pages;
  while (static_cast<int>(pg.size()) > keep) {
    release_page(pt, pg.back());
    pg.pop_back();
    row[pg.size()] = -1;
  }
  pt->capacity[slot] = keep * pt->page_size;
  const int st = write_row_range(pt, slot, keep, had - keep);
  if (st != PKV_OK) return st;
  return pkv::ok();
}

// With U pages in use, those numbered above U move to the free pages among
// 1..U, both taken in ascending order.
int pt_compact(pkv_pt *pt, int32_t *pairs_out, int max_pairs, int *n_pairs) {
  if (!pt || !n_pairs) return pkv::fail(PKV_E_BAD_ARG, "pt_compact: NULL");
  const int used = pt->n_pages - 1 - static_cast<int>(pt->free_pages.size());
  int moves = 0;
  for (int p = used + 1; p < pt->n_pages; ++p) moves += pt->refs[p] > 0;
  *n_pairs = moves;
  if (!pairs_out) return pkv::ok();   // the count alone
  if (max_pairs < moves)
    return pkv::fail(PKV_E_BAD_ARG, "pt_compact: room for %d pairs needed", moves);
  std::vector<int32_t> to;
  try {
    to.assign(pt->n_pages, 0);
  } catch (...) {
    return pkv::fail(PKV_E_BAD_ARG, "pt_compact: out of host memory");
  }
  int dst = 1, n = 0;
  for (int p = used + 1; p < pt->n_pages; ++p) {
    if (pt->refs[p] == 0) continue;
    while (pt->refs[dst] != 0) ++dst;   // as many free pages below as used ones above
    to[p] = dst;
    pt->refs[dst] = pt->refs[p];
    pt->refs[p] = 0;
    pairs_out[2 * n] = p;
    pairs_out[2 * n + 1] = dst;
    ++n;
  }
  for (int s = 1; s < pt->n_slots; ++s) {
    int32_t *row = pt->table.data() + static_cast<size_t>(s) * pt->max_pages;
    for (size_t b = 0; b < pt->pages[s].size(); ++b) {
      const int32_t p = pt->pages[s][b];
      if (to[p]) pt->pages[s][b] = row[b] = to[p];
    }
  }
  pt->free_pages.clear();   // its room was reserved when the table was made
  for (int p = pt->n_pages - 1; p > used; --p) pt->free_pages.push_back(p);
  if (n > 0) {
    const int st = write_row_range(pt, 0, 0, 1LL * pt->n_slots * pt->max_pages);
    if (st != PKV_OK) return st;
  }
  return pkv::ok();
}

int pt_page_refs(const pkv_pt *pt, int page, int *n) {
  if (!pt || !n) return pkv::fail(PKV_E_BAD_ARG, "pt_page_refs: NULL");
  if (page < 0 || page >= pt->n_pages)
    return pkv::fail(PKV_E_BAD_ARG, "pt_page_refs: page %d out of range", page);
  *n = pt->refs[page];
  return pkv::ok();
}

int pt_capacity(const pkv_pt *pt, int slot, int *tokens) {
  if (!pt || !tokens) return pkv::fail(PKV_E_BAD_ARG, "pt_capacity: NULL");
  if (slot < 0 || slot >= pt->n_slots)
    return pkv::fail(PKV_E_BAD_SLOT, "pt_capacity: slot %d out of range", slot);
  *tokens = pt->capacity[slot];
  return pkv::ok();
}

int pt_pages(const pkv_pt *pt, int slot, int32_t *host_out, int max, int *n) {
  if (!pt || !n) return pkv::fail(PKV_E_BAD_ARG, "pt_pages: NULL");
  if (slot < 0 || slot >= pt->n_slots)
    return pkv::fail(PKV_E_BAD_SLOT, "pt_pages: slot %d out of range", slot);
  const auto &pg = pt->pages[slot];
  *n = static_cast<int>(pg.size());
  if (host_out)
    for (int i = 0; i < *n && i < max; ++i) host_out[i] = pg[i];
  return pkv::ok();
}

int pt_free_pages(const pkv_pt *pt, int *n) {
  if (!pt || !n) return pkv::fail(PKV_E_BAD_ARG, "pt_free_pages: NULL");
  *n = static_cast<int>(pt->free_pages.size());
  return pkv::ok();
}

int pt_free_page_list(const pkv_pt *pt, int32_t *host_out, int max, int *n) {
  if (!pt || !n) return pkv::fail(PKV_E_BAD_ARG, "pt_free_page_list: NULL");
  *n = static_cast<int>(pt->free_pages.size());
  if (host_out)
    for (int i = 0; i < *n && i < max; ++i) host_out[i] = pt->free_pages[i];
  return pkv::ok();
}

int pt_host_table(const pkv_pt *pt, int32_t *host_out, int max) {
  if (!pt || !host_out) return pkv::fail(PKV_E_BAD_ARG, "pt_host_table: NULL");
  int n = static_cast<int>(pt->table.size());
  if (max < n)
    return pkv::fail(PKV_E_BAD_ARG, "pt_host_table: need %d entries", n);
  std::copy(pt->table.begin(), pt->table.end(), host_out);
  return pkv::ok();
}

}  // extern "C"
