"""Paged cache, without a GPU: the ends of the ranges, what the binding keeps
between calls, and the host-side parts of the kernels' bookkeeping (every
pointer below is fake and never dereferenced).
"""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import paged as P
from test_paged_host import _attend, _desc, _lib, _read, _write


def test_rows_that_a_loop_of_32_bits_cannot_count_are_refused():
    """Sq * Hq from 2^31 - 2^15 on: a row index steps past its last value."""
    b, L = _lib()
    for Sq, Hq in ((16383, 131079), (13902, 154473), (16383, 131088)):
        assert (1 << 31) - (1 << 15) <= Sq * Hq
        d = _desc(b, B=1, Sq=Sq, Hq=Hq, d=32)
        assert L.pi_attn_paged_workspace_bytes(ctypes.byref(d)) == 0
        assert _attend(L, d) == b.PI_ERR_UNSUPPORTED


def test_rows_to_read_past_32_bits_are_refused():
    """From 2^31 - 2^15 on, rounding Sq up to whole CTAs would wrap."""
    b, L = _lib()
    for Sq in ((1 << 31) - 1, (1 << 31) - (1 << 15)):
        assert _read(L, _desc(b, Sq=Sq)) == b.PI_ERR_UNSUPPORTED
        assert _write(L, _desc(b, Sq=Sq)) == b.PI_ERR_UNSUPPORTED
        assert _attend(L, _desc(b, Sq=Sq)) == b.PI_ERR_UNSUPPORTED


STAGE_CHECK = r"""
#include <cstdio>
#include "stage.h"
using piattn::Stuck;

// A barrier as try_wait.parity sees it: done(p) holds once the phase of parity p
// before the one under way is complete.
struct Bar {
  int issued = 0, landed = 0;
  bool done(unsigned p) const { return ((unsigned)landed & 1u) != p; }
};

// The warp's loop over `tiles` tiles, stopped at the wait for K (which 0) or V (1)
// of tile `at`.  Whether the parities handed back wait for every copy under way.
static bool waits_for_all(int tiles, int at, int which) {
  Bar k, v;
  k.issued = v.issued = 1;
  Stuck stuck = Stuck::kNo;
  unsigned used = 0;
  for (int i = 0; i < tiles; ++i) {
    const bool more = i + 1 < tiles;
    if (i == at && which == 0) { stuck = Stuck::kAtK; break; }
    k.landed = k.issued;
    if (more) ++k.issued;
    if (i == at && which == 1) { stuck = more ? Stuck::kAtVAhead : Stuck::kAtV; break; }
    v.landed = v.issued;
    ++used;
    if (more) ++v.issued;
  }
  const piattn::StagePhases last = piattn::last_phases(used, stuck);
  // a wait must not be over while a copy is under way, and must end with it
  const bool k_open = k.issued > k.landed, v_open = v.issued > v.landed;
  if (k_open == k.done(last.k) || v_open == v.done(last.v)) return false;
  k.landed = k.issued;
  v.landed = v.issued;
  return k.done(last.k) && v.done(last.v);
}

int main() {
  for (int tiles = 1; tiles < 9; ++tiles)
    for (int at = 0; at < tiles; ++at)
      for (int which = 0; which < 2; ++which)
        if (!waits_for_all(tiles, at, which)) {
          std::printf("tile %d of %d, wait %d\n", at, tiles, which);
          return 1;
        }
  std::printf("stage ok\n");
}
"""


def test_a_stopped_warp_waits_for_its_last_copies(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "stage.cc", tmp_path / "stage"
    src.write_text(STAGE_CHECK)
    csrc = os.path.join(ROOT, "vla_prefix_lm_b200", "csrc")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "stage ok" in r.stdout, r.stdout


# -------------------------------------------- what the binding keeps between calls

def _descriptor(b, **kw):
    """The descriptor that a call with these arguments would pass."""
    pages = torch.empty(4, 16, 1, 256, dtype=torch.bfloat16)
    table = torch.empty(2, 3, dtype=torch.int32)
    return b._paged_desc(2, 5, 8, torch.bfloat16, pages, table, **kw)[2]


def test_a_scale_changed_in_place_is_a_new_scale(monkeypatch):
    b, _ = _lib()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    scale, window, sinks = torch.tensor(0.5), torch.tensor(7), np.array(3)
    d = _descriptor(b, softmax_scale=scale, window=window, sinks=sinks)
    assert (d.softmax_scale, d.window, d.sinks) == (0.5, 7, 3)
    scale.mul_(0.5)
    window.add_(2)
    sinks += 1
    d = _descriptor(b, softmax_scale=scale, window=window, sinks=sinks)
    assert (d.softmax_scale, d.window, d.sinks) == (0.25, 9, 4)
    assert _descriptor(b, softmax_scale=0.25, window=9, sinks=4) is d


def test_refusals_do_not_depend_on_earlier_calls(monkeypatch):
    b, _ = _lib()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for _ in range(2):
        _descriptor(b, window=2, sinks=1)
        for bad in (dict(window=2.0, sinks=1), dict(window=2, sinks=1.0),
                    dict(window=torch.tensor(2.0), sinks=1)):
            with pytest.raises(TypeError):
                _descriptor(b, **bad)
        with pytest.raises(ValueError):
            _descriptor(b, window=2 ** 31, sinks=1)
        with pytest.raises((TypeError, ValueError)):
            _descriptor(b, softmax_scale="wide")


# ------------------------------------------------------ the stated rounding bounds

@pytest.mark.parametrize("top", [224.0001, 225.0, 256.0, 300.0, 447.9, 448.0])
@pytest.mark.parametrize("e", [-125, -126, -20, 0, 17, 119, 120])
def test_the_headers_rounding_bounds(top, e):
    """The larger of 2^-4 of the value (half a step of 2^-3 * 2^k for scaled values in
    [2^k, 2^(k+1)), k >= -6) and 2^-10 of the scale (half of the subnormals' step,
    2^-9); 224 * 2^-13 > 2^-6, so the former from 2^-13 of the largest on."""
    if top * 2.0 ** e >= 2.0 ** 128:
        pytest.skip("past the largest float")
    x = np.concatenate([[top], top * np.exp2(np.linspace(-16, 0, 20001))]) * 2.0 ** e
    vals, byte = P.quantise(x)
    assert byte == e + 127
    err, scale = np.abs(vals * 2.0 ** e - x), 2.0 ** e
    near = x >= 2.0 ** -13 * x[0]
    assert (err[near] <= 2.0 ** -4 * x[near]).all()
    assert (err <= np.maximum(2.0 ** -4 * x, 2.0 ** -10 * scale)).all()
    if top < 230:                      # and not from 2^-14 on: e4m3 is subnormal there
        far = x >= 2.0 ** -14 * x[0]
        assert (err[far] > 2.0 ** -4 * x[far]).any()


@pytest.mark.parametrize("top", [1e-44, 1e-40, 1.1754943508222875e-38, 1e-36])
def test_the_bounds_where_the_exponent_stops(top):
    x = top * np.linspace(0, 1, 1001)
    vals, byte = P.quantise(x)
    assert byte == 1
    scale = 2.0 ** -126
    err = np.abs(vals * scale - x)
    assert (err <= np.maximum(2.0 ** -4 * x, 2.0 ** -10 * scale)).all()


def test_a_zero_vector_has_scale_one():
    vals, byte = P.quantise(np.zeros(4))
    assert byte == 127 and (vals == 0).all()


# ------------------------------------------------------------------ a C client

def test_plain_c_client_and_the_descriptors_layout(tmp_path):
    b, _ = _lib()
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    exe, libdir = tmp_path / "paged_check", os.path.join(ROOT, "vla_prefix_lm_b200")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c_abi", "paged_check.c"),
                    "-L", libdir, "-lpiattn", f"-Wl,-rpath,{libdir}", "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.split("\n")
    assert "c abi ok" in lines
    got = {w[0]: tuple(map(int, w[1:])) for w in map(str.split, lines) if len(w) == 3 and w[0] != "c"}
    want = {}
    for name, _ in b.PiPagedDesc._fields_:
        field = getattr(b.PiPagedDesc, name)
        want[name] = (field.offset, field.size)
    assert got == want
    assert f"size {ctypes.sizeof(b.PiPagedDesc)}" in lines
