"""The block manager when the host runs out of memory: a step's calls return a
status (no exception leaves a C entry) and leave the books whole.  A small
program replaces operator new and lets its n-th allocation fail, for every n."""

import os
import shutil
import subprocess

import pytest

from paged_kv_cache_473_b200 import build as bld

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include "block_manager.h"

static long left = -1;  // allocations until one fails; below 0: none does
static void* get(std::size_t n) {
  if (left >= 0 && left-- == 0) throw std::bad_alloc();
  if (void* p = std::malloc(n)) return p;
  throw std::bad_alloc();
}
void* operator new(std::size_t n) { return get(n); }
void* operator new[](std::size_t n) { return get(n); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
void operator delete[](void* p) noexcept { std::free(p); }
void operator delete[](void* p, std::size_t) noexcept { std::free(p); }

#define NEED(x) do { if (!(x)) { std::printf("line %d, allocation %ld: %s\n", __LINE__, n, #x); return 1; } } while (0)

static const int kBlocks = 1200;
static int64_t ids[kBlocks];

// Sequences 0 (known, then drafts), 1 (a fork) and many of one block each.
static pa_block_manager* books() {
  pa_block_manager* bm = pa_bm_create(kBlocks, 2);
  pa_bm_add_sequence(bm, 0, ids, 3, nullptr);
  int64_t seq = 0, slot;
  int32_t cow[2], k;
  for (int i = 0; i < 5; ++i) pa_bm_append_slots(bm, &seq, nullptr, 1, &slot, cow, &k);
  pa_bm_fork(bm, 0, 1);
  for (int i = 2; i < 1100; ++i) pa_bm_add_sequence(bm, i, nullptr, 1, nullptr);
  return bm;
}

static bool whole(pa_block_manager* bm) {  // every block is free or held
  int held = 0;
  for (int b = 0; b < kBlocks; ++b) held += pa_bm_ref_count(bm, b) > 0;
  return held + pa_bm_num_free(bm) == kBlocks;
}

int main() {
  for (int i = 0; i < kBlocks; ++i) ids[i] = i;
  for (long n = 0; n < 40; ++n) {
    pa_block_manager* bm = books();
    left = n;
    pa_status_t st = pa_bm_truncate(bm, 0, 6, ids + 3, 3);
    left = -1;
    NEED(st == PA_OK && pa_bm_length(bm, 0) == 6 && whole(bm));
    left = n;  // many blocks come back
    for (int i = 2; i < 1100; ++i)
      if ((st = pa_bm_free_sequence(bm, i)) != PA_OK) break;
    left = -1;
    NEED(st == PA_OK && whole(bm));
    int64_t seqs[2] = {0, 1}, tok[2] = {6, 9}, slots[2];
    int32_t cow[4], k = 0;
    int free_before = pa_bm_num_free(bm);
    left = n;
    st = pa_bm_append_slots(bm, seqs, tok, 2, slots, cow, &k);
    left = -1;
    if (st == PA_OK)
      NEED(pa_bm_length(bm, 0) == 7 && pa_bm_length(bm, 1) == 9);
    else
      NEED(st == PA_ERR_INVALID && pa_bm_length(bm, 0) == 6 && pa_bm_length(bm, 1) == 8 && pa_bm_num_free(bm) == free_before);
    NEED(whole(bm));
    NEED(pa_bm_append_slots(bm, seqs, tok, 2, slots, cow, &k) == PA_OK && whole(bm));
    NEED(pa_bm_free_sequence(bm, 0) == PA_OK && pa_bm_free_sequence(bm, 1) == PA_OK);
    NEED(pa_bm_num_free(bm) == kBlocks);
    pa_bm_destroy(bm);
  }
  std::puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_no_allocation_that_fails_ends_the_process_or_loses_a_block(tmp_path):
    src = tmp_path / "books.cpp"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "books")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(bld.ROOT, "include"), str(src),
                    os.path.join(bld.CSRC, "block_manager.cpp"), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert got.returncode == 0 and got.stdout == "ok\n", (got.returncode, got.stdout, got.stderr)
