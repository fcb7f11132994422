"""Which kernels the GPU tests of the operators reach, checked on the CPU.

linear_i8 chooses a kernel, a tile and the parts of K by fitted times, and the
attention the parts of the keys; a refit moves the sizes at which they change.
The choices are host code of post_pruning_b200/csrc, compiled here into a small
program (nothing runs on a GPU) that is asked about the sizes of the GPU tests.
"""

import os
import subprocess

import pytest

import test_gpu_attention
import test_gpu_attention_parts
import test_gpu_attention_units
import test_gpu_linear_i8
from test_host_plans import CSRC, ROOT, _nvcc

HARNESS = r'''
#include <cstdio>
#include <cstring>
#include "FILE"

namespace sgpt {
void count_launches(unsigned long long) {}
long long wait_limit_cycles() { return kDefaultWaitCycles; }
}

int main() {
  using namespace sgpt;
  long long n, seqs, heads, kv, width, d, rows;
  (void)n, (void)seqs, (void)heads, (void)kv, (void)width, (void)d, (void)rows;
  ASK
  return 0;
}
'''
LINEAR = r'''
  while (scanf("%lld %lld %lld", &n, &d, &rows) == 3) {
    const Plan p = plan((int)rows, (int)n, (int)d);
    printf("%d %d %d\n", (int)p.pair, p.bn, p.split);
  }
'''
ATTENTION = r'''
  while (scanf("%lld %lld %lld %lld %lld", &n, &seqs, &heads, &kv, &width) == 5) {
    const bool pair = heads / kv % 2 == 0;
    const int parts = parts_for(n, (int)seqs, (int)(pair ? heads / 2 : heads), pair, (int)width);
    printf("%d %d %lld\n", (int)pair, parts, attention_ctas(n, (int)seqs, (int)heads, (int)kv));
  }
'''


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """ask(file, questions): a tuple of numbers for each."""
    if _nvcc() is None:
        pytest.skip("nvcc not found")
    where, built = tmp_path_factory.mktemp("plans"), {}

    def answer(file, questions):
        if file not in built:
            src, exe = where / (file + ".host.cu"), where / (file + ".exe")
            src.write_text(HARNESS.replace("FILE", file).replace("ASK", LINEAR if "linear" in file else ATTENTION))
            r = subprocess.run([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O2", "-std=c++17", "-I" + CSRC,
                                "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                               capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            built[file] = exe
        r = subprocess.run([str(built[file])], input="\n".join(" ".join(map(str, q)) for q in questions),
                           capture_output=True, text=True, timeout=60)
        assert r.returncode == 0
        out = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(out) == len(questions)
        return out

    return answer


def _cases(test, names):
    """The values of a parametrised test's argument names, as tuples."""
    for mark in test.pytestmark:
        if mark.name == "parametrize" and mark.args[0] == names:
            return [tuple(v) for v in mark.args[1]]
    raise AssertionError(names)


PLANS = {(1, bn, split) for bn in (128, 256) for split in (1, 2)} | {(0, bn, split) for bn in (16, 32, 64)
                                                                    for split in (1, 2, 4, 8)}


def _plans_of(ask, *tests):
    sizes = [s for t in tests for s in _cases(t, "n,d_in,d_out")]
    return set(ask("linear_i8.cu", sizes))


def test_linear_i8_values_are_checked_for_every_plan(ask):
    m = test_gpu_linear_i8
    reached = _plans_of(ask, m.test_linear_i8, m.test_linear_i8_every_variant, m.test_linear_i8_pairs_on_128_tokens,
                        m.test_linear_i8_wide_tiles_with_k_split)
    assert reached == PLANS, PLANS - reached


def test_linear_i8_timeouts_are_checked_for_every_kind(ask):
    """Of each kernel, its tiles alone and with K in parts."""
    m = test_gpu_linear_i8
    reached = _plans_of(ask, m.test_linear_i8_wait_times_out, m.test_linear_i8_pairs_on_128_tokens,
                        m.test_linear_i8_wide_tiles_with_k_split)
    kinds = {(pair, bn if pair else 0, split > 1) for pair, bn, split in reached}
    assert kinds == {(1, 128, False), (1, 128, True), (1, 256, False), (1, 256, True), (0, 0, False), (0, 0, True)}, kinds


def _attention_of(ask, lens, shapes):
    return ask("attention.cu", [(sum(lens), len(lens), *s) for s in shapes])


def test_attention_units_are_taken_from_other_ctas(ask):
    """The tests of taken units run unsplit launches of several times as many
    CTAs as there are SMs, of both kinds of unit and both widths."""
    m = test_gpu_attention_units
    for (heads, kv, width), (pair, parts, ctas) in zip(m.SHAPES, _attention_of(ask, m.LENS, m.SHAPES)):
        assert parts == 1 and ctas >= 3 * 148, (heads, kv, width, parts, ctas)
    assert {(heads // kv % 2, width) for heads, kv, width in m.SHAPES} == {(0, 64), (0, 128), (1, 64), (1, 128)}


def test_attention_values_are_checked_for_every_part_count(ask):
    """Each number of parts of the keys, of both kinds of unit and both widths."""
    reached = set()
    for m, test in ((test_gpu_attention, test_gpu_attention.test_attention),
                    (test_gpu_attention_parts, test_gpu_attention_parts.test_parts)):
        for lens, heads, kv in _cases(test, "lens,heads,kv"):
            for width in (64, 128):
                (pair, parts, _), = _attention_of(ask, lens, [(heads, kv, width)])
                reached.add((pair, parts, width))
    want = {(pair, parts, width) for pair in (0, 1) for parts in (1, 2, 4, 8) for width in (64, 128)}
    assert reached == want, want - reached
