// Page tables of a paged KV cache on the host: reference counts, copy on
// write, lowest free page first (include/mk.h, mk_pages_*). Every call checks
// everything it needs before it changes anything, and reserves its memory
// first, so that a failing call leaves the object as it was.
#include <algorithm>
#include <cstring>
#include <exception>
#include <vector>

#include "mk_ops.h"

using namespace mk;

struct mk_pages {
  int n_blocks = 0, block_size = 0, n_seqs = 0, capacity = 0, entries = 0;
  std::vector<int32_t> refs;     // [n_blocks] sequences that hold the page
  std::vector<int32_t> table;    // [n_seqs][entries], -1: none
  std::vector<int32_t> length;   // [n_seqs]
  std::vector<uint64_t> free_bits;  // bit set: the page is free
  // within mk_pages_resize: a copy of the call reads the page, so that it is not
  // free before the call is over (a copy into it could run first)
  std::vector<uint8_t> held;     // [n_blocks]
  int n_free = 0;
  int first = 0;                 // no free page lies in a word below this one

  int used(int length_) const { return (length_ + block_size - 1) / block_size; }
  int take() {
    int w = first;
    while (!free_bits[w]) ++w;
    first = w;
    const int b = w * 64 + __builtin_ctzll(free_bits[w]);
    free_bits[w] &= free_bits[w] - 1;
    refs[b] = 1;
    --n_free;
    return b;
  }
  void give(int b) {
    if (--refs[b] == 0 && !held[b]) {
      free_bits[b / 64] |= 1ull << (b % 64);
      first = std::min(first, b / 64);
      ++n_free;
    }
  }
  // the pages that the call's copies read, free now if nobody holds them
  void release(const std::vector<int32_t>& sources) {
    for (int32_t b : sources) {
      if (!held[b]) continue;  // a second copy of the same page
      held[b] = 0;
      if (refs[b] == 0) {
        refs[b] = 1;
        give(b);
      }
    }
  }
};

extern "C" {

int mk_pages_create(int n_blocks, int block_size, int n_seqs, int kv_capacity, mk_pages** out) {
  if (!out) return op_fail(MK_ERR_INVALID, "out is NULL");
  *out = nullptr;
  if (n_blocks < 1 || block_size < 1 || n_seqs < 1 || kv_capacity < 1)
    return op_fail(MK_ERR_INVALID,
                   "n_blocks, block_size, n_seqs and kv_capacity must be at least 1");
  if ((int64_t)kv_capacity + block_size > INT32_MAX)
    return op_fail(MK_ERR_INVALID, "kv_capacity + block_size must fit 31 bits");
  mk_pages* p = nullptr;
  try {
    p = new mk_pages();
    p->n_blocks = n_blocks;
    p->block_size = block_size;
    p->n_seqs = n_seqs;
    p->capacity = kv_capacity;
    p->entries = p->used(kv_capacity);
    p->refs.assign(n_blocks, 0);
    p->held.assign(n_blocks, 0);
    p->table.assign((size_t)n_seqs * p->entries, -1);
    p->length.assign(n_seqs, 0);
    p->free_bits.assign((size_t)n_blocks / 64 + 1, 0);
    for (int b = 0; b < n_blocks; ++b) p->free_bits[b / 64] |= 1ull << (b % 64);
    p->n_free = n_blocks;
  } catch (const std::exception&) {
    delete p;
    return op_fail(MK_ERR_OOM, "no host memory for the page tables");
  }
  *out = p;
  return MK_OK;
}

int mk_pages_destroy(mk_pages* p) {
  delete p;
  return MK_OK;
}

int mk_pages_resize(mk_pages* p, int n, const int32_t* seqs, const int32_t* lengths,
                    mk_block_copy* copies, int capacity, int* n_copies) {
  if (!p || !n_copies || n < 0 || (n > 0 && (!seqs || !lengths)) || capacity < 0 ||
      (capacity > 0 && !copies))
    return op_fail(MK_ERR_INVALID, "mk_pages_resize: a NULL or negative argument");
  *n_copies = 0;
  // First the whole call without taking a page: whether a partly filled page is
  // shared, and how many pages are free, depends on the sequences before it in
  // the list. The counts it lowers are written down and raised again.
  std::vector<uint8_t> seen;
  std::vector<int32_t> lowered, sources;
  const char* why = nullptr;
  int code = MK_ERR_INVALID, made = 0;
  try {
    seen.assign(p->n_seqs, 0);
    size_t most = 0;
    for (int i = 0; i < n; ++i)
      if (seqs[i] >= 0 && seqs[i] < p->n_seqs) most += (size_t)p->used(p->length[seqs[i]]);
    lowered.reserve(most);
    sources.reserve(std::min(n, p->n_seqs));
  } catch (const std::exception&) {
    return op_fail(MK_ERR_OOM, "no host memory");
  }
  int free_now = p->n_free;
  for (int i = 0; i < n && !why; ++i) {
    const int s = seqs[i], len = lengths[i];
    if (s < 0 || s >= p->n_seqs) why = "sequence out of range [0, n_seqs)";
    else if (len < 0 || len > p->capacity) why = "length out of range [0, kv_capacity]";
    else if (seen[s]) why = "a sequence is named twice";
    if (why) break;
    seen[s] = 1;
    const int32_t* t = &p->table[(size_t)s * p->entries];
    const int old = p->length[s], u0 = p->used(old), u1 = p->used(len);
    if (len > old) {
      free_now -= u1 - u0;
      if (old % p->block_size && p->refs[t[u0 - 1]] > 1) {
        --free_now;
        ++made;
        --p->refs[t[u0 - 1]];
        lowered.push_back(t[u0 - 1]);
        p->held[t[u0 - 1]] = 1;
        sources.push_back(t[u0 - 1]);
      }
      if (free_now < 0) {
        why = "not enough free pages";
        code = MK_ERR_OOM;
      }
    } else {
      for (int e = u1; e < u0; ++e) {
        if (--p->refs[t[e]] == 0 && !p->held[t[e]]) ++free_now;
        lowered.push_back(t[e]);
      }
    }
  }
  for (int32_t b : lowered) ++p->refs[b];
  if (!why && made > capacity) why = "copies: capacity is too small";
  if (why) {
    p->release(sources);
    return op_fail(code, why);
  }

  for (int i = 0; i < n; ++i) {
    int32_t* t = &p->table[(size_t)seqs[i] * p->entries];
    const int old = p->length[seqs[i]], u0 = p->used(old), u1 = p->used(lengths[i]);
    if (lengths[i] > old) {
      if (old % p->block_size && p->refs[t[u0 - 1]] > 1) {
        const int mine = p->take(), shared = t[u0 - 1];
        p->give(shared);
        t[u0 - 1] = mine;
        copies[(*n_copies)++] = {shared, mine, old % p->block_size};
      }
      for (int e = u0; e < u1; ++e) t[e] = p->take();
    } else {
      for (int e = u1; e < u0; ++e) {
        p->give(t[e]);
        t[e] = -1;
      }
    }
    p->length[seqs[i]] = lengths[i];
  }
  p->release(sources);
  return MK_OK;
}

int mk_pages_fork(mk_pages* p, int n, const int32_t* parents, const int32_t* children) {
  if (!p || n < 0 || (n > 0 && (!parents || !children)))
    return op_fail(MK_ERR_INVALID, "mk_pages_fork: a NULL or negative argument");
  std::vector<uint8_t> child;
  try {
    child.assign(p->n_seqs, 0);
  } catch (const std::exception&) {
    return op_fail(MK_ERR_OOM, "no host memory");
  }
  for (int i = 0; i < n; ++i) {
    if (parents[i] < 0 || parents[i] >= p->n_seqs || children[i] < 0 || children[i] >= p->n_seqs)
      return op_fail(MK_ERR_INVALID, "sequence out of range [0, n_seqs)");
    if (p->length[children[i]] != 0 || child[children[i]])
      return op_fail(MK_ERR_INVALID, "a child must be an empty sequence, named once");
    child[children[i]] = 1;
  }
  for (int i = 0; i < n; ++i)
    if (child[parents[i]])
      return op_fail(MK_ERR_INVALID, "a sequence is both a parent and a child");
  for (int i = 0; i < n; ++i) {
    const int32_t* t = &p->table[(size_t)parents[i] * p->entries];
    int32_t* c = &p->table[(size_t)children[i] * p->entries];
    const int u = p->used(p->length[parents[i]]);
    for (int e = 0; e < u; ++e) ++p->refs[c[e] = t[e]];
    p->length[children[i]] = p->length[parents[i]];
  }
  return MK_OK;
}

int mk_pages_compact(mk_pages* p, mk_block_copy* copies, int capacity, int* n_copies) {
  if (!p || !n_copies || capacity < 0 || (capacity > 0 && !copies))
    return op_fail(MK_ERR_INVALID, "mk_pages_compact: a NULL or negative argument");
  *n_copies = 0;
  const int live = p->n_blocks - p->n_free;
  int need = 0;
  for (int b = live; b < p->n_blocks; ++b) need += p->refs[b] > 0;
  if (need > capacity) {
    *n_copies = need;
    return op_fail(MK_ERR_INVALID, "copies: capacity is too small");
  }
  if (need == 0) return MK_OK;
  std::vector<int32_t> moved;  // new number of each page from `live` on
  try {
    moved.assign(p->n_blocks - live, -1);
  } catch (const std::exception&) {
    return op_fail(MK_ERR_OOM, "no host memory");
  }
  for (int b = live; b < p->n_blocks; ++b) {
    if (p->refs[b] == 0) continue;
    const int to = p->take();  // below `live`: as many are free there as are in use above
    p->refs[to] = p->refs[b];
    p->refs[b] = 1;
    p->give(b);
    moved[b - live] = to;
    copies[(*n_copies)++] = {b, to, p->block_size};
  }
  for (int s = 0; s < p->n_seqs; ++s) {
    int32_t* t = &p->table[(size_t)s * p->entries];
    for (int e = 0; e < p->used(p->length[s]); ++e)
      if (t[e] >= live) t[e] = moved[t[e] - live];
  }
  return MK_OK;
}

int mk_pages_read(const mk_pages* p, int32_t* tables, int32_t* lengths, int* n_free) {
  if (!p) return op_fail(MK_ERR_INVALID, "pages is NULL");
  if (tables) std::memcpy(tables, p->table.data(), p->table.size() * sizeof(int32_t));
  if (lengths) std::memcpy(lengths, p->length.data(), p->length.size() * sizeof(int32_t));
  if (n_free) *n_free = p->n_free;
  return MK_OK;
}

}  // extern "C"
