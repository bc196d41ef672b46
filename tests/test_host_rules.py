"""Host rules of the launches (csrc/host.cuh), compiled with the host compiler and run here."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routed_expert_ffn_route_gb300", "csrc")


def run_cpp(tmp_path, body):
    """What a program prints whose main() is `body`."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include "host.cuh"\n#include <cstdio>\n#include <vector>\nint main() {\n'
                   + body + "\n}\n")
    cxx = shutil.which("g++") or shutil.which("c++")
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o",
                        str(exe), "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()


def test_answers_are_kept_by_device(tmp_path):
    out = run_cpp(tmp_path, """
  moe::DeviceAnswers a;
  int asked = 0;
  auto q = [&](int dev, int what) {
    return a.get(dev, what, [&]() { asked++; return 100 * (dev + 1) + what; });
  };
  printf("%d %d %d ", q(0, 8), q(1, 8), q(0, 4));
  printf("%d %d %d ", q(1, 8), q(0, 8), q(0, 4));
  printf("%d", asked);""")
    assert out == ["108", "208", "104", "208", "108", "104", "3"]


@pytest.mark.parametrize("failure", [0, -1])
def test_a_failed_query_is_asked_again(tmp_path, failure):
    out = run_cpp(tmp_path, f"""
  moe::DeviceAnswers a;
  int asked = 0;
  auto q = [&]() {{ return a.get(0, 8, [&]() {{ return asked++ ? 18 : {failure}; }}); }};
  printf("%d ", q());
  printf("%d ", q());
  printf("%d ", q());
  printf("%d", asked);""")
    assert out == [str(failure), "18", "18", "2"]


def test_the_products_plan_asks_through_them():
    """lin_clusters keeps its answers by device and split, and no failed one."""
    with open(os.path.join(CSRC, "linear.cu")) as f:
        src = f.read()
    body = src[src.index("static int lin_clusters("):]
    body = body[:body.index("\n}\n")]
    assert "static DeviceAnswers" in body and "known.get(dev, split," in body
    assert "std::atomic" not in src


@pytest.mark.parametrize("n,refused,tried,status", [
    (1, 99, "1", 0), (2048, 99, "1", 0), (2049, 99, "8", 0), (32768, 99, "8", 0),
    (32769, 99, "16", 0), (1048560, 99, "16", 0),
    (1048560, 16, "16 8", 0),        # no room for sixteen CTAs: eight
    (1048560, 8, "16 8", 7), (4096, 8, "8", 7), (1, 1, "1", 7)])
def test_sort_falls_back_to_eight_ctas(tmp_path, n, refused, tried, status):
    """Launches of `refused` CTAs or more fail."""
    out = run_cpp(tmp_path, f"""
  const int e = moe::sort_launch({n}, [](int ctas) {{
    printf("%d ", ctas);
    return ctas >= {refused} ? 7 : 0;
  }});
  printf("%d", e);""")
    assert out == tried.split() + [str(status)]


def test_the_sort_launches_through_it():
    with open(os.path.join(CSRC, "tokens.cu")) as f:
        src = f.read()
    assert src.count("sort_launch(n, [&](int ctas)") == 1
    assert src.count("cudaLaunchKernelEx(&cfg, sort_tokens_kernel") == 1
