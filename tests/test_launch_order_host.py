"""What a stream's last launch leaves for the next one to wait for (csrc/launch_order.h,
built for the host). No GPU needed."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "decode_attention_kv_dattn_gb300", "csrc")

SHIM = r'''
#include <cstdio>
#include <cstdlib>
#include "launch_order.h"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)
int main() {
  dattn::LaunchOrder o;
  int a, b, s, t;  // caches, streams
  CHECK(!o.writes(&s, &a) && !o.in_order(&s));
  o.record(&s, &a);
  CHECK(o.writes(&s, &a) && !o.writes(&s, &b) && !o.writes(&t, &a) && !o.in_order(&s));
  // results that may be the next call's inputs: the next launch on the stream starts behind them, and only that one
  o.record_results(&s);
  CHECK(!o.writes(&s, &a) && o.in_order(&s) && !o.in_order(&t));
  CHECK(o.in_order(&s));  // (a launch that failed leaves it so)
  o.started(&s);
  CHECK(!o.in_order(&s));
  o.record(&s, nullptr);
  CHECK(!o.in_order(&s) && !o.writes(&s, &a) && !o.writes(&s, nullptr));
  // a call of several launches: the first of them takes it
  o.record_results(&s);
  o.record_results(&t);
  o.started(&s);
  o.record(&s, &b);
  CHECK(!o.in_order(&s) && o.writes(&s, &b) && o.in_order(&t));
  std::printf("ok\n");
  return 0;
}
'''


def test_order(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "shim.cpp", str(tmp_path / "shim")
    src.write_text(SHIM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.stdout.strip() == "ok", r.stdout
