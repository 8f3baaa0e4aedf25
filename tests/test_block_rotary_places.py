"""Where rotary's outputs may lie: what shares a place with another tensor's input,
with the other output or with itself is refused on the host; the same tensors, and
slices of one buffer, are not."""

import os
import shutil
import subprocess

import pytest
import torch

from test_block_boundary import CSRC, FAKE, needs_lib
from test_block_linear_boundary import E, b, rotary_args

BF16 = torch.bfloat16


def at(offset, sb=2560, sl=256, sh=64):
    """(2, 10, heads, 64) bf16, `offset` values from the stand-in address on."""
    return FAKE + 2 * offset, sb, sl, sh


FAR = 1 << 20
# valid: everything apart, k with two heads
APART = dict(q=at(0), k=at(FAR), q_out=at(2 * FAR), k_out=at(3 * FAR))


@needs_lib
@pytest.mark.parametrize("over", [
    dict(q_out=at(FAR), k_out=at(0)),                           # out = (k, q)
    dict(q_out=at(FAR)),                                        # q's results over k
    dict(k_out=at(0)),
    dict(q=at(FAR), q_out=at(FAR)),                             # q and k are one tensor, turned in place
    dict(q_out=at(64)),                                         # q, a head further on
    dict(q_out=at(0, sb=5120)), dict(q_out=at(0, sh=128, sl=512)),      # q's place, other strides
    dict(k_out=at(FAR, sl=128)), dict(q_out=at(2560)),          # the next sample
    dict(k_out=at(2 * FAR)), dict(k_out=at(2 * FAR + 64)),      # both outputs
    dict(q_out=at(2 * FAR, sh=32)), dict(q_out=at(2 * FAR, sl=8)), dict(k_out=at(3 * FAR, sb=0)),    # within itself
    dict(k_out=at(3 * FAR, sb=256 * 9)),
    # slices of one buffer of eight heads, one head too many
    dict(q=at(0, 5120, 512), q_out=at(192, 5120, 512)),
    # unequal strides that cross: q's heads 200 apart, q_out's 72
    dict(q=at(0, 1 << 15, 1024, 200), q_out=at(8, 1 << 15, 1024, 72)),
])
def test_places_that_meet_are_refused(over):
    args = rotary_args(**dict(APART, **over))
    assert b._lib().muon_rotary(args, None) == E.MUON_E_ARG
    text = b._lib().muon_block_last_error()
    assert b"overlap" in text or b"place" in text


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_places_against_every_value(tmp_path):
    """Small layouts against the places of all their values; those of the tensors
    that a call may be given, and sizes past 64 bits of bytes, by hand."""
    src = tmp_path / "p.cpp"
    src.write_text("""
#include "block_overlap.h"
#include <cstdio>
#include <random>
#include <set>
using namespace muon;
int main() {
  std::mt19937 g(1);
  auto pick = [&](int n) { return int64_t(g() % unsigned(n)); };
  auto all = [](const Places& p, bool& twice) {
    std::set<int64_t> s;
    twice = false;
    for (int64_t i = 0; i < p.count[0]; ++i) for (int64_t j = 0; j < p.count[1]; ++j)
    for (int64_t k = 0; k < p.count[2]; ++k) for (int64_t l = 0; l < p.count[3]; ++l)
      if (!s.insert((int64_t)(uintptr_t)p.ptr / 2 + i * p.stride[0] + j * p.stride[1] + k * p.stride[2] + l * p.stride[3]).second) twice = true;
    return s;
  };
  int bad = 0, met = 0, apart = 0, repeats = 0;
  for (int t = 0; t < 60000; ++t) {
    Places a{}, b{};
    const bool same = pick(2);
    for (Places* p : {&a, &b}) {
      p->ptr = (void*)(uintptr_t)(4000 + 2 * pick(60));
      for (int i = 0; i < 4; ++i) {
        p->count[i] = pick(20) ? 1 + pick(4) : 0;
        p->stride[i] = i == 3 ? 1 : pick(6) ? 1 + pick(pick(2) ? 12 : 60) : 0;
        if (p == &b && same) p->stride[i] = a.stride[i];
      }
    }
    bool ta, tb;
    const auto sa = all(a, ta), sb = all(b, tb);
    bool meet = false;
    for (int64_t v : sa) meet = meet || sb.count(v);
    bad += places_meet(a, b, 2) != meet;
    bad += places_meet(b, a, 2) != meet;
    bad += places_repeat(a) != ta;
    meet ? ++met : ++apart;
    repeats += ta;
  }
  const int64_t n = 1024, h = 16, d = 128, l = 3 * h * d;
  char* base = (char*)(uintptr_t)(1 << 20);
  auto view = [&](int64_t first, int64_t sb, int64_t sl, int64_t sh, int64_t heads) {
    return Places{base + 2 * first, {sb, sl, sh, 1}, {16, n, heads, d}};
  };
  const Places q = view(0, n * l, l, d, h), k = view(h * d, n * l, l, d, h), late = view(1, n * l, l, d, h);
  const Places few = view(h * d, n * l, l, d, 4), more = view((h + 4) * d, n * l, l, d, 4), heads_first = view(0, 2 * n * h * d, d, n * d, h);
  const Places next = view(n * h * d, 2 * n * h * d, h * d, d, h);
  bad += places_meet(q, k, 2) || places_meet(k, few, 2) != true || places_meet(few, more, 2) || places_repeat(q) || !places_meet(q, late, 2);
  bad += places_meet(heads_first, next, 2) || places_repeat(heads_first);
  const int64_t top = int64_t(1) << 40, many = 0x7fffffff;
  const Places far{base, {top, top, top, 1}, {many, 1, 2, d}}, other{base + 2 * d, {top, top, top, 1}, {many, 1, 1, d}};
  bad += !places_repeat(far) || places_meet(far, other, 2) || !places_meet(far, far, 2) || places_repeat(other);
  // a layout that no one writes out: steps of 2 and 4 cannot make up 1, and there are too many ways to try them all
  const Places even{base, {6, 4, 2, 1}, {many, many, many, 1}}, odd{base + 2, {8, 10, 2, 1}, {many, many, many, 1}};
  bad += !places_meet(even, odd, 2);
  printf("bad %d met %d apart %d repeats %d\\n", bad, met, apart, repeats);
}
""")
    exe = tmp_path / "p"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split()
    assert got[1] == "0" and all(int(got[i]) > 5000 for i in (3, 5, 7)), got
    assert os.path.exists(os.path.join(CSRC, "block_overlap.h"))


@pytest.mark.gpu
def test_slices_of_one_buffer():
    """q, k and both outputs inside one buffer, in place or beside each other, with
    as many key heads as query heads and fewer; what overlaps raises and leaves
    everything as it was."""
    import matrix_aware_optimizer_periodic_amd as m
    gen = torch.Generator(device="cuda").manual_seed(0)
    for n in (1, 7):
        for h, g in ((4, 4), (4, 1)):
            both = h + g
            buf = torch.randn(3, n, 2 * both, 64, generator=gen, device="cuda").to(BF16)
            f = m.rotary_freqs(48)
            q, k, to_q, to_k = buf.split((h, g, h, g), dim=2)
            want = m.rotary_fwd(q.contiguous(), k.contiguous(), f, offset=5)
            before = buf.clone()
            m.rotary_fwd(q, k, f, offset=5, out=(to_q, to_k))
            assert torch.equal(to_q, want[0]) and torch.equal(to_k, want[1]) and torch.equal(buf[:, :, :both], before[:, :, :both])
            first = buf.clone()
            bad = [(k, q)] if h == g else []
            bad += [(buf[:, :, 1:1 + h], to_k), (to_q, buf[:, :, h - 1:both - 1]), (to_q, buf[:, :, both:both + g]),
                    (q, buf[:, :, :g])]
            for out in bad:
                with pytest.raises((m.MuonError, ValueError)):
                    m.rotary_fwd(q, k, f, offset=5, out=out)
            with pytest.raises(m.MuonError):
                m.rotary_fwd(q, q, f, offset=5, out=(q, to_q))
            torch.cuda.synchronize()
            assert torch.equal(buf, first)
            m.rotary_fwd(q, k, f, offset=5, out=(q, k))
            assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(buf[:, :, both:], first[:, :, both:])
