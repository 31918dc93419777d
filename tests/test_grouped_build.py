"""What the grouped kernels' build and first call check: the registers that a kernel starts with, and device
properties that are kept only where they were found (CPU only)."""
import glob
import os
import subprocess

import pytest

from bit_quantized_moe_route_b200 import build

LOG = "ptxas info    : 0 bytes gmem\nptxas info    : Used {} registers, used 1 barriers\n"


def gu(name):
    return os.path.join(build.CSRC, f"gu_{name}.cu")


def test_every_form_has_its_count():
    counts = {os.path.basename(s): build.launch_registers(s) for s in build.sources()}
    forms = {k: v for k, v in counts.items() if k.startswith("gu_")}
    assert len(forms) == len(glob.glob(os.path.join(build.CSRC, "gu_*.cu"))) >= 15
    assert all(v is None for k, v in counts.items() if not k.startswith("gu_"))
    for name, regs in forms.items():
        whole = name in ("gu_mm.cu", "gu_dx.cu", "gu_dw.cu")      # one MMA per step, sums in tensor memory
        assert regs == (None if whole else 96 if "_any" in name else 168), name


@pytest.mark.parametrize("name,good", [("mm_wide", 168), ("dw_f32", 162), ("fp8_any", 96), ("dx_any", 90)])
def test_registers_are_checked(name, good):
    build.check_registers(gu(name), LOG.format(good))
    for bad in (good - 8, good + 8, 255):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_registers(gu(name), LOG.format(bad))
    with pytest.raises(RuntimeError, match="registers"):
        build.check_registers(gu(name), "")
    build.check_registers(gu("mm"), LOG.format(40))               # shares nothing out
    build.check_registers(os.path.join(build.CSRC, "moe_api.cu"), LOG.format(40))


def test_a_count_that_does_not_fit_fails_the_build(monkeypatch, tmp_path):
    """The compile step itself refuses, and leaves no object behind."""
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path))
    obj = tmp_path / "gu_mm_wide.cu.o"

    class Run:
        returncode, stdout = 0, LOG.format(128)

    def nvcc(cmd, **kw):
        assert "-v" in cmd
        obj.write_bytes(b"")
        return Run

    monkeypatch.setattr(build.subprocess, "run", nvcc)
    with pytest.raises(RuntimeError, match="128"):
        build._compile(gu("mm_wide"), False)
    assert not obj.exists()


CACHE = """
#include "device_cache.h"
#include <cstdio>
int main() {
  static moe::DeviceCache c;
  int asked = 0, answer = -1;
  auto query = [&] { ++asked; return answer; };
  bool ok = c.get(3, query) == -1 && c.get(3, query) == -1 && asked == 2;   // a failure is not kept
  answer = 0;
  ok = ok && c.get(3, query) == 0 && asked == 3;
  answer = 74;
  ok = ok && c.get(3, query) == 74 && asked == 4;
  answer = 5;
  ok = ok && c.get(3, query) == 74 && asked == 4;                           // what was found is
  ok = ok && c.get(2, query) == 5 && asked == 5;                            // for its device
  ok = ok && c.get(64, query) == 5 && c.get(64, query) == 5 && asked == 7;  // beyond those kept
  std::puts(ok ? "ok" : "bad");
}
"""


def test_failed_queries_are_asked_again(tmp_path):
    src = tmp_path / "cache.cpp"
    src.write_text(CACHE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, "-o", str(tmp_path / "cache"), str(src)],
                   check=True)
    assert subprocess.run([str(tmp_path / "cache")], capture_output=True, text=True, check=True).stdout.strip() == "ok"
