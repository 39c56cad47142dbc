"""The dense layers' plan (csrc/dense_plan.h, host code, compiled here by itself): no shape takes a kernel that none of
the tested shapes takes, so that new costs cannot drop a kernel out of the tests or bring an untested one in."""
import os
import random
import shutil
import subprocess

import pytest

from dense_shapes import CASES, products

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "dense_plan.h"
#include <stdio.h>
using namespace tw;
int main() {
  int bf16, kind, dual, M, N, batch;
  long long K;
  for (int T = 1; T <= 256; ++T)            // rows that a thread adds up for the column sums
    for (int cols = 8; cols <= 1 << 20; cols *= 2)
      for (int join = 0; join < 2; ++join)
        printf("# %d %d %d %d\n", T, cols, join, (strip_of(T, true, join) + 7) / (narrow_strip(T, cols, join) ? 32 : 8));
  while (scanf("%d %d %d %d %d %lld %d", &bf16, &kind, &dual, &M, &N, &K, &batch) == 7) {
    const Split p = split_of(bf16, kind, dual, M, N, K, batch);
    printf("%d %d %d %d %d\n", p.cls, p.S, p.ks, (int)p.planes, sum_blocks(bf16, kind, p, N));
  }
}
"""
KINDS, CLASSES = ("along", "across", "both"), ("small", "mid", "large", "narrow", "deep")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "activation_sparse_transformer_up_amd", "csrc"),
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def ask(rows):
        """(class, S, ks, planes, blocks of column sums) of every (bf16, kind, dual, M, N, K, batch)."""
        text = "".join("%d %d %d %d %d %d %d\n" % r for r in rows)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        lines = out.splitlines()
        ask.strips = [tuple(map(int, line[1:].split())) for line in lines if line[0] == "#"]
        return [tuple(map(int, line.split())) for line in lines if line[0] != "#"]
    return ask


def kernels(plan, cases):
    """Per case, the kernels of its products: type, kind, one, dual or batch, tile, planes, whether k is split."""
    rows = [[(int(t == "bf16"), *p) for p in products(op, T, K, N, lay)] for op, T, K, N, t, lay in cases]
    answers = iter(plan([r for c in rows for r in c]))
    out = []
    for c in rows:
        out.append(set())
        for b, kind, dual, *_, batch in c:
            cls, S, _, planes, _ = next(answers)
            out[-1].add(("bf16" if b else "f32", KINDS[kind], "dual" if dual else "batch" if batch > 1 else "one", CLASSES[cls],
                         "planes" if planes else "plain", "split" if S > 1 else "whole"))
    return out


def shapes(seed, n):
    rng = random.Random(seed)

    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))
    for _ in range(n):
        op = rng.choice(["linear", "linear_back", "gated", "gated_back"])
        yield op, log(1, 20000), 8 * log(1, 1800 if op.startswith("linear") else 520), 8 * log(1, 1800), rng.choice(["bf16", "f32"]), rng.choice(
            ["nk", "kn"])


def test_every_kernel_is_tested(plan):
    tested = set().union(*kernels(plan, CASES))
    met = {}
    for case, ks in zip((all_shapes := list(shapes(1, 100000))), kernels(plan, all_shapes)):
        for k in ks:
            met.setdefault(k, case)
    missing = {k: c for k, c in met.items() if k not in tested}
    assert not missing, missing
    # nothing of the tiles is out of reach: single, dual and three-fold products, all classes, planes
    for k in (("bf16", "across", "one", "deep", "plain", "split"), ("bf16", "along", "dual", "mid", "plain", "whole"),
              ("bf16", "along", "dual", "narrow", "plain", "split"), ("f32", "along", "one", "narrow", "plain", "split"),
              ("f32", "along", "dual", "narrow", "plain", "split"), ("f32", "across", "one", "mid", "planes", "split"),
              ("f32", "along", "dual", "mid", "planes", "whole"), ("bf16", "both", "batch", "large", "plain", "split")):
        assert k in tested and k in met, k


def test_splits_cover_k(plan):
    """S ranges of ks, a multiple of 64, hold all of k and none is empty; at most 64, their sums within 256 MB."""
    cases = list(shapes(2, 3000))
    rows = [(int(t == "bf16"), *p) for op, T, K, N, t, lay in cases for p in products(op, T, K, N, lay)]
    for (b, kind, dual, M, N, K, batch), (cls, S, ks, planes, blocks) in zip(rows, plan(rows)):
        assert ks % 64 == 0 and 1 <= S <= 64 and (S - 1) * ks < K <= S * ks
        assert S == 1 or S * batch * M * (1 + dual) * N * 4 <= 256 << 20
        assert not (b and planes) and blocks >= 1


def test_few_fp32_rows_fit_their_places(plan):
    """The 128 x 32 tile takes 80 KB of LDS, two per CU: its splits stay within the 512 places that there are."""
    rng = random.Random(5)
    rows = [(0, 0, dual, 8 * rng.randint(1, 1800), rng.randint(1, 32), 8 * rng.randint(8, 1800), 1) for _ in range(3000) for dual in (0, 1)]
    seen = 0
    for (_, _, dual, M, N, K, _), (cls, S, _, planes, _) in zip(rows, plan(rows)):
        if CLASSES[cls] == "narrow" and S > 1:
            seen += 1
            assert -(-M * (1 + dual) // 128) * S <= 512, (M, N, K, S)
    assert seen > 100


def test_column_sums_of_few_rows(plan):
    """A thread adds up at most 8 rows of up to 256, 4 where each row is itself a sum over the splits of k, unless the
    columns alone fill the CUs."""
    plan([])
    assert len(plan.strips) == 256 * 18 * 2
    for T, cols, join, rows in plan.strips:
        if cols < 65536:
            assert rows <= (4 if join else 8), (T, cols, join, rows)
