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


SHIM_KEYS = r'''
#include <cstdio>
#include <cstdlib>
#include <set>
#include <thread>
#include "launch_order.h"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)
int main() {
  using dattn::stream_key;
  int s, cache, other;
  auto h = [](uintptr_t x) { return reinterpret_cast<const void*>(x); };
  CHECK(stream_key(&s, 0) == stream_key(&s, 5));
  // the legacy default stream (handles 0 and 1) of each device; the per-thread one (2) of each thread besides
  for (int d = 0; d < 8; ++d) {
    CHECK(stream_key(h(0), d) == stream_key(h(1), d) && stream_key(h(0), d) != stream_key(h(2), d));
    for (int e = 0; e < d; ++e) CHECK(stream_key(h(0), d) != stream_key(h(0), e) && stream_key(h(2), d) != stream_key(h(2), e));
  }
  const void *mine = stream_key(h(2), 0), *theirs = nullptr, *legacy = nullptr;
  CHECK(mine == stream_key(h(2), 0));
  std::thread t([&] { theirs = stream_key(h(2), 0), legacy = stream_key(h(0), 0); });
  t.join();
  CHECK(theirs && theirs != mine && legacy == stream_key(h(0), 0));
  // an append on one device's default stream is not forgotten for a decode on another's
  dattn::LaunchOrder o;
  o.record(stream_key(h(0), 0), &cache);
  o.record(stream_key(h(0), 1), &other);
  CHECK(o.writes(stream_key(h(0), 0), &cache) && o.writes(stream_key(h(0), 1), &other));
  std::printf("ok\n");
  return 0;
}
'''


def test_default_streams_of_devices_and_threads(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "shim.cpp", str(tmp_path / "shim")
    src.write_text(SHIM_KEYS)
    subprocess.run([cxx, "-O1", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.stdout.strip() == "ok", r.stdout
