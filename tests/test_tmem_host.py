"""TMEM columns without a cycle of waits, shown on the host.

tcgen05.alloc waits until its columns are free, without a limit.  A launch that
programmatic serialisation starts early keeps the columns it gets until the launch before
it has ended, so that one must own all of its columns by then: a kernel lets its dependents
start only behind the barrier after its allocation (one call of a block is enough to
let them)."""
import glob
import os
import re
import subprocess

import pytest

from linear_forms import FORMS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_ffn_06_b200", "csrc")


def _kernels_with_tmem():
    """(file, name, body) of every kernel that allocates TMEM."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in text.split("__global__")[1:]:
            body = part[:part.find("\n}\n")]
            if "tmem_alloc" in body:
                name = re.search(r"(\w+_kernel)\(", body).group(1)
                found.append((os.path.basename(path), name, body))
    return found


def test_the_kernels_with_tmem_are_found():
    assert [(f, n) for f, n, _ in _kernels_with_tmem()] == [
        ("decode_tc.cu", "decode_tc_kernel"), ("gemm_tc.cu", "grouped_gemm_kernel"),
        ("linear_i8.cu", "linear_i8_kernel")]


@pytest.mark.parametrize("kernel", _kernels_with_tmem(), ids=lambda k: k[1])
def test_dependents_start_behind_the_allocation(kernel):
    body = kernel[2]
    alloc = max(m.start() for m in re.finditer(r"tmem_alloc", body))
    owned = body.index("tmem_base = ctl->tmem_base")
    barrier = body.rindex("__syncthreads()", 0, owned)  # the barrier that publishes the columns
    triggers = [m.start() for m in re.finditer(r"pdl_trigger\(\)", body)]
    assert alloc < barrier and triggers and min(triggers) > owned


# Blocks on an SM together ask for no more columns than it has.  What a plan of the int8
# product takes is counted here from the sizes of an SM, not from the library's own rule:
# the system's 1 KB and the dynamic shared memory alone (static adds to it).
SWEEP = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "linear_plan.cuh"
using namespace moe;
int main() {
  const long long SM = 228 * 1024;
  std::vector<long long> Ts, Ns, Ks;
  for (int t = 1; t <= 130; ++t) Ts.push_back(t);
  for (long long t : {160, 192, 255, 256, 257, 300, 511, 512, 600, 1000, 1024, 1030, 4096, 9999,
                      16384, 1000000, (1 << 24) - 1}) Ts.push_back(t);
  for (long long k : {16, 48, 128, 144, 256, 400, 512, 1040, 2048, 2816, 4096, 4112, 8192, 14336,
                      131056}) Ks.push_back(k);
  for (long long n : {1, 7, 64, 130, 500, 1000, 2816, 4096, 9000, 14336, 28672, 40000, 128256,
                      (1 << 22) - 1}) Ns.push_back(n);
  struct Seen { int cols; long long smem; };
  std::vector<Seen> seen;  // per number of columns the smallest block
  for (int sms : {148, 132})
    for (int fit : {1, 0})
      for (int gated : {0, 1})
        for (long long T : Ts) for (long long N : Ns) for (long long K : Ks) {
          const int NO = gated ? (int)(N + 1) / 2 : (int)N;
          const LinPlan p = plan_linear(T, NO, (int)K, gated != 0, sms, [&](int s) {
            return fit ? (s == 8 ? 15 : 33) : 0; });
          if (p.few || p.blocks == 0) continue;
          auto bad = [&](const char* what) {
            printf("%s: T %lld NO %d K %lld gated %d\n", what, T, NO, K, gated); exit(1); };
          const long long rows = gated ? 64 : 128, stage = 128 * 128 + p.tn / p.cg * 128 * p.nsub;
          if (p.stages < 1 || p.stages > kMaxStages) bad("stages");
          if ((long long)p.smem < 1024 + p.stages * stage) bad("ring");
          if (p.split > 1 && (long long)p.smem < 1024 + (p.tn + 31) / 32 * 32 * 512) bad("sums");
          if (p.smem + kLinStatic > 227 * 1024) bad("too much shared memory");
          if (p.tn % (16 * p.cg) || p.tn < 16 || p.tn > 256) bad("columns of an MMA");
          const int used = p.nbuf * p.nsub == 2 ? 256 + p.tn : (p.tn + 31) / 32 * 32;
          if (used > (int)p.cols || p.nbuf * p.nsub > 2) bad("columns");
          if (p.MT * p.cg * rows < NO || (long long)p.TT * p.nsub * p.tn < T) bad("cover");
          if (p.split > 1 && (p.KB < p.split || p.blocks != (int)(p.MT * p.TT))) bad("split");
          bool found = false;
          for (Seen& s : seen)
            if (s.cols == (int)p.cols) {
              found = true;
              if ((long long)p.smem + 1024 < s.smem) s.smem = p.smem + 1024;
            }
          if (!found) seen.push_back({(int)p.cols, (long long)p.smem + 1024});
        }
  // the other kernels with TMEM: expert products and decode products, their smallest
  for (auto s : {Seen{512, 214704}, Seen{128, 92000}, Seen{64, 90000}}) seen.push_back(s);
  // the most columns that blocks of any kinds sharing an SM ask for
  std::vector<int> most(SM / 16 + 1, 0);
  for (long long m = 0; m <= SM / 16; ++m)
    for (const Seen& s : seen) {
      const long long rest = m - (s.smem + 15) / 16;
      if (rest >= 0 && most[rest] + s.cols > most[m]) most[m] = most[rest] + s.cols;
    }
  for (const Seen& s : seen) printf("%d columns: %lld bytes\n", s.cols, s.smem);
  printf("columns asked for together: %d\n", most[SM / 16]);
  return most[SM / 16] > 512;
}
"""


def test_blocks_that_share_an_sm_share_its_columns(tmp_path):
    src, exe = tmp_path / "sweep.cpp", tmp_path / "sweep"
    src.write_text(SWEEP)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, "-x", "c++", "-o", str(exe), str(src)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr


PLAN = r"""
#include <cstdio>
#include <cstdlib>
#include "linear_plan.cuh"
int main(int n, char** v) {
  for (int i = 1; i + 2 < n; i += 3) {
    const moe::LinPlan p = moe::plan_linear(atoll(v[i]), atoi(v[i + 1]) / 2, atoi(v[i + 2]), true, 148,
                                            [](int s) { return s == 8 ? 15 : 33; });
    printf("%d %d %d %d %d\n", p.few, p.cg, p.split, p.ew, p.nsub);
  }
}
"""


def test_the_sizes_that_stand_for_a_form_reach_it(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PLAN)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, "-x", "c++", "-o", str(exe), str(src)])
    out = subprocess.check_output([str(exe), *(str(n) for size in FORMS for n in size)], text=True)
    got = [tuple(int(n) for n in line.split()) for line in out.splitlines()]
    assert got == [(0, *form) for form in FORMS.values()]
