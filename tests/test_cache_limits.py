"""Calls at the edges of what the cache operators' contract allows, as far as the CPU
can tell: sizes, build, the host's arithmetic (no GPU needed)."""

from __future__ import annotations

import importlib.util
import itertools
import os
import re
import subprocess
import textwrap

import pytest
import torch

from exact_attention_63_gb300 import build, cache
from test_cache_abi import ARCH, SCALE, WORKSPACE, L, a_cache, calls, tokens  # noqa: F401


@pytest.mark.parametrize("group", [1, 2, 3, 4, 7, 8, 16, 33, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_a_workspace_serves_every_smaller_call(L, group, d):  # noqa: F811
    """The size for a max_seqlen is enough for each call of no larger max_seqlen, and where
    total is the smaller: the device is reached (here: missing)."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls would reach it")
    sizes = [cache.workspace_size(2 * group, 2, m, d) for m in range(1, cache.MAX_NEW + 1)]
    assert sizes == sorted(sizes)
    for most, total in itertools.product((1, 2, 9, 16, 17, 20, 33, 40, 65, 100, 128), (1, 8, 16, 18, 30, 32, 60, 128)):
        run = calls(L, a_cache(d=d), tokens(total=total, max_seqlen=most, H=2 * group), ws_bytes=sizes[most - 1])
        assert run["attend"]() == ARCH, (most, total)
    run = calls(L, a_cache(d=d), tokens(total=128, max_seqlen=1, H=2 * group), ws_bytes=sizes[0] - 1)
    assert run["attend"]() == WORKSPACE


@pytest.mark.parametrize("source,loaders", [("cache_attn.cu", 1), ("cache_weights.cu", 2)])
def test_a_loader_waits_for_its_copies_whatever_ended_it(source, loaders):
    """A copy that lands in shared memory after its CTA has ended lands in another CTA's.  Where only the
    consumer's wait ran out the loader has seen nothing of it, so its last waits depend on no flag."""
    with open(os.path.join(build.CSRC, source)) as f:
        text = f.read()
    waits = re.findall(r"if \(([^\n]*)\) \{[^\n]*\n\s*const uint64_t t0 = globaltimer_ns\(\);\n(?:\s*auto drain|\s*for \(int i = max)",
                       text)
    assert waits == ["lane == 0"] * loaders


@pytest.fixture
def fake_build(monkeypatch, tmp_path):
    """build.build() whose commands only leave their output file: (commands run, paths of the outputs)."""
    ran = []

    def run(cmd, what, verbose=False):
        ran.append(what)
        open(cmd[cmd.index("-o") + 1], "w").close()

    paths = {"LIB_PATH": str(tmp_path / "lib.so"), "BIND_PATH": str(tmp_path / "bind.so"), "BUILD_DIR": str(tmp_path / "o")}
    for name, path in paths.items():
        monkeypatch.setattr(build, name, path)
    monkeypatch.setattr(build, "run", run)
    monkeypatch.setattr(build, "nvcc_path", lambda: "/cuda/bin/nvcc")
    return ran, paths


def test_the_library_is_built_without_torch(fake_build, monkeypatch, capsys):
    ran, paths = fake_build
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == paths["LIB_PATH"]
    assert os.path.exists(paths["LIB_PATH"]) and not os.path.exists(paths["BIND_PATH"])
    assert "link" in ran and not any("bind" in what for what in ran)
    assert "PyTorch" in capsys.readouterr().err


def test_a_binding_that_does_not_build_leaves_the_library(fake_build, monkeypatch):
    ran, paths = fake_build
    run = build.run

    def fails(cmd, what, verbose=False):
        if "bind" in what:
            raise RuntimeError("no compiler")
        run(cmd, what, verbose)

    monkeypatch.setattr(build, "run", fails)
    with pytest.raises(RuntimeError, match="no compiler"):
        build.build()
    assert os.path.exists(paths["LIB_PATH"]) and not os.path.exists(paths["BIND_PATH"])


def test_both_are_built(fake_build):
    ran, paths = fake_build
    assert build.build() == paths["LIB_PATH"]
    assert all(os.path.exists(paths[name]) for name in ("LIB_PATH", "BIND_PATH"))
    assert ran.index("link") < ran.index("link of the binding")


def test_a_binding_for_another_torch_is_refused(L, monkeypatch):  # noqa: F811
    monkeypatch.setattr(cache, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.raises(RuntimeError, match="built for PyTorch"):
        cache._load()
    assert cache._bind is None
    monkeypatch.undo()
    assert cache._load() is cache._bind


def test_weights_refuse_scales_that_no_lse_can_be_divided_by(L):  # noqa: F811
    """-LSE/scale has to fit into 32 bits: of LSE = 7 it does not at 1e-38."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls would reach it")
    for scale, expect in ((1e-38, SCALE), (9.9e-31, SCALE), (1.1e-30, ARCH), (1e30, ARCH)):
        assert calls(L, a_cache(), tokens(), scale=scale)["weigh"]() == expect, scale


def test_division_by_multiplication(tmp_path):
    """FastDiv over the ends of its range: each divisor's multiples and their neighbours up to 2^31 - 1."""
    source, program = tmp_path / "div.cpp", tmp_path / "div"
    source.write_text(textwrap.dedent("""
        #include <cstdio>
        #include "cache_launch.h"
        int main() {
          const long long top = 0x7FFFFFFF;
          long long bad = 0, n = 0;
          auto check = [&](int d) {
            const attn::FastDiv f = attn::fast_div(d);
            auto at = [&](long long x) {
              if (x < 0 || x > top) return;
              ++n;
              bad += f(static_cast<int>(x)) != x / d;
            };
            for (long long q = 0; q < 40; ++q)
              for (int e = -2; e <= 2; ++e) {
                at(q * d + e);
                at((top / d - q) * d + e);
                at(top - q);
                at((1ll << (q % 31)) + e);
              }
          };
          for (int d = 1; d < 70000; ++d) check(d);
          for (int b = 16; b < 31; ++b)
            for (int e = -3; e <= 3; ++e) check((1 << b) + e);
          check(top);
          check(top - 1);
          std::printf("%lld of %lld\\n", bad, n);
          return bad != 0;
        }
    """))
    include = os.path.join(build.cuda_home(build.nvcc_path()), "include")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + include, "-I" + build.CSRC, str(source), "-o", str(program)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
