"""The plans of the forms that the GPU tests run, by the library's own planner (CPU only: a small host program
that links the library): a form that has moved to another kernel would leave its own untested."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "bit_diffusion_model_svdq_amd"))
import build  # noqa: E402  (the package's build script: compiler and folders)

from tests.attention_forms import FORMS, TOKENS, sizes  # noqa: E402
from tests.rope_forms import CASES, launch_of  # noqa: E402

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "svdq_internal.h"
int main() {
  std::printf("%d\n", svdq::device_cu_count());
  char kind[16];
  while (std::scanf("%15s", kind) == 1) {
    if (!std::strcmp(kind, "attention")) {
      svdq::SpanArgs a = {};
      if (std::scanf("%d %d %d %d %d %d %d %d %d %d %d", &a.batch, &a.total_q, &a.total_k, &a.heads_q, &a.heads_kv,
                     &a.head_dim, &a.causal, &a.left, &a.right, &a.sinks, &a.prefix) != 11) return 1;
      const svdq::SpanPlan p = svdq::plan_attention_spans(a);
      const int waves = !p.own.keys ? p.own.waves : p.wide || a.head_dim <= 64 ? 4 : 2;
      std::printf("%s %d %d %d %d %d %d\n", p.own.keys ? "keys" : "rows", waves, p.own.parts, p.own.splits,
                  p.pre_splits, p.own.chunk, p.tail_splits);
    } else {
      svdq::QkNormRopeArgs a = {};
      long long rows;
      if (std::scanf("%lld %d %d %d", &rows, &a.heads_q, &a.heads_k, &a.head_dim) != 4) return 1;
      a.rows = rows;
      std::printf("%lld\n", (long long)svdq::qk_norm_rope_blocks(a));
    }
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if not os.path.exists(build.HIPCC) and not shutil.which("hipcc"):
        pytest.skip("hipcc not available")
    folder = tmp_path_factory.mktemp("plans")
    src, exe = folder / "plans.cpp", folder / "plans"
    src.write_text(PROGRAM)
    r = subprocess.run([build.HIPCC, "-x", "hip", "--cuda-host-only", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                        build.CSRC, str(src), "-x", "none", build.LIB, f"-Wl,-rpath,{build.PKG}", "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]

    def ask(kind, args):
        line = f"{kind} {' '.join(map(str, args))}\n"
        r = subprocess.run([str(exe)], input=line, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        cus, answer = r.stdout.splitlines()
        if cus != "256":
            pytest.skip("planned for 256 compute units")
        return answer.split()

    return ask


@pytest.mark.parametrize("form", FORMS)
def test_forms(plans, form):
    *call, want = FORMS[form]
    kernel, *numbers = plans("attention", sizes(*call))
    assert (kernel, *map(int, numbers[:4])) == want
    assert int(numbers[5]) == 0


@pytest.mark.parametrize("form", TOKENS)
def test_new_tokens(plans, form):
    """Also that no share is longer than the chain of sums that the tolerance counts."""
    *call, want, chain = TOKENS[form]
    kernel, *numbers = plans("attention", sizes(*call))
    assert (kernel, *map(int, numbers[:4])) == want
    splits, pre, chunk = (int(numbers[i]) for i in (2, 3, 4))
    prefix = 0 if isinstance(call[6], tuple) else call[6]
    if pre:
        assert chunk <= chain and -(-prefix // chunk) <= pre and -(-max(call[1]) // chunk) <= splits
    elif splits > 1:
        assert chunk <= chain and -(-(sum(call[6]) + 3) // chunk) <= splits
    else:
        seen = max(call[1])
        if prefix:
            seen += prefix
        elif call[6][0] >= 0:
            seen = min(seen, sum(call[6]) + 3)
        assert seen <= chain


@pytest.mark.parametrize("case", CASES, ids=str)
def test_steps_of_norm_and_rotation(plans, case):
    """The launch has the workgroups of the steps that the case is there for, and not of fewer; more steps
    than its workgroups need a wave never takes."""
    lens, hq, hk, d, steps = case
    blocks = int(plans("rope", (sum(lens), hq, hk, d))[0])
    assert blocks == launch_of(sum(lens), hq, hk, d, steps)
    assert all(launch_of(sum(lens), hq, hk, d, n) != blocks for n in range(1, steps))
