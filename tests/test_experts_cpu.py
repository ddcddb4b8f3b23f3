"""The expert-layer calls without a GPU: the library exports what experts.h
declares, bad arguments get their status before any device call, and the kernels
keep their working set out of scratch memory."""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from partitioned_chip_accumulation_amd import build, experts, hist

OK, BAD, UNSUPPORTED = hist.HIST_OK, hist.HIST_ERR_INVALID_ARG, hist.HIST_ERR_UNSUPPORTED
P = 4096  # a plausible, aligned address that no call here reads


def test_header_and_binding_agree():
    text = open(os.path.join(build.INCLUDE, "experts.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = {m.group(1): m.group(2).count(",") + 1
                for m in re.finditer(r"hist_status_t (experts_\w+)\(([^)]*)\)", text)}
    bound = {k: len(v) for k, v in experts._SIGNATURES.items()}
    assert declared == bound
    lib = ctypes.CDLL(hist.LIBRARY)
    assert all(hasattr(lib, name) for name in declared)
    assert int(re.search(r"EXPERTS_MAX_EXPERTS (\d+)u", text).group(1)) == experts.MAX_EXPERTS
    assert int(re.search(r"EXPERTS_MAX_TOP_K (\d+)u", text).group(1)) == experts.MAX_TOP_K


def calls(name, good, bad):
    """Each of the (position, value) changes of the good arguments is refused."""
    fn = getattr(experts._library(), name)
    for at, value in bad:
        args = list(good)
        args[at] = value
        assert fn(*args, None) == BAD, (name, at, value)


def test_argument_errors_before_any_device_call():
    lib = experts._library()
    n = ctypes.c_uint64(0)
    size = lib.experts_group_workspace_size
    assert size(100, 8, 256, ctypes.byref(n)) == OK and n.value == 0
    assert size(65536, 8, 256, ctypes.byref(n)) == OK and n.value % (256 * 4) == 0 and n.value
    assert size(100, 0, 256, ctypes.byref(n)) == BAD
    assert size(100, 8, 0, ctypes.byref(n)) == BAD
    assert size(100, 8, 256, None) == BAD
    assert size(100, 8, 1025, ctypes.byref(n)) == UNSUPPORTED
    assert size(100, 65, 256, ctypes.byref(n)) == UNSUPPORTED
    assert size(2**40, 8, 256, ctypes.byref(n)) == UNSUPPORTED
    assert size(2**64 - 1, 64, 256, ctypes.byref(n)) == UNSUPPORTED

    calls("experts_group", (P, 32, 100, 8, 256, P, P, P, P, None, 0),
          [(0, None), (0, P + 2), (1, 16), (3, 0), (4, 0), (5, None), (6, None), (7, None),
           (8, None), (5, P + 1), (7, P + 2)])
    big = (P, 32, 65536, 8, 256, P, P, P, P)
    for ws, bytes_ in ((None, 2**30), (P, 1024), (P + 2, 2**30)):
        assert lib.experts_group(*big, ws, bytes_, None) == hist.HIST_ERR_WORKSPACE

    calls("experts_matmul", (P, 64, P, 128, 10, P, 128, 8192, P, P, 20, 2, 4, 64, 128, 0),
          [(0, None), (0, P + 1), (1, 63), (2, None), (3, 127), (4, 0), (5, None), (6, 127),
           (7, -1), (8, None), (8, P + 2), (9, P + 2), (9, None), (11, 0), (12, 0), (13, 0),
           (14, 0), (15, 2), (15, -1)])
    calls("experts_matmul_dx", (P, 128, P, 64, P, 128, 8192, P, 20, 4, 64, 128, 0),
          [(0, None), (1, 127), (2, None), (3, 63), (4, None), (5, 127), (6, -1), (7, None),
           (9, 0), (10, 0), (11, 0), (12, 5)])
    calls("experts_matmul_dw", (P, P, 64, P, 128, 10, P, P, 20, 2, 4, 64, 128, 0),
          [(0, None), (0, P + 1), (1, None), (2, 63), (3, None), (4, 127), (5, 0), (6, None),
           (7, None), (9, 0), (10, 0), (11, 0), (12, 0), (13, 2)])
    calls("experts_combine", (P, 64, P, 64, 20, P, P, 10, 2, 64, 0),
          [(0, None), (1, 63), (2, None), (3, 63), (5, None), (6, P + 1), (8, 0), (9, 0), (10, 2)])
    calls("experts_combine_backward", (P, 64, P, P, 64, P, 64, P, P, P, 10, 2, 64, 0),
          [(0, None), (1, 63), (2, None), (3, None), (4, 63), (5, None), (6, 63), (7, None),
           (8, None), (9, None), (11, 0), (12, 0), (13, 2)])
    calls("experts_quantize_rows", (P, 64, P, P, 64, 10, 64, 0),
          [(0, None), (1, 63), (2, None), (3, None), (3, P + 1), (4, 63), (6, 0), (7, 2)])
    calls("experts_int8_matmul",
          (P, 64, P, 128, 10, P, P, 128, 8192, P, P, P, 20, 2, 4, 64, 128, 0),
          [(0, None), (1, 63), (2, None), (3, 127), (4, 0), (5, None), (6, None), (7, 127),
           (8, -1), (9, None), (10, None), (11, None), (13, 0), (14, 0), (15, 0), (16, 0),
           (17, 2)])
    # sizes beyond the documented limits
    assert lib.experts_matmul(P, 64, P, 128, 10, P, 128, 8192, P, P, 2**31, 2, 4, 64, 128, 0,
                              None) == UNSUPPORTED
    assert lib.experts_quantize_rows(P, 2**18, P, P, 2**18, 10, 2**18, 0, None) == UNSUPPORTED
    assert lib.experts_combine(P, 64, P, 64, 20, P, P, 2**60, 2, 64, 0, None) == UNSUPPORTED


def test_header_is_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    source = tmp_path / "c.c"
    source.write_text("#include \"experts.h\"\nint main(void) { return experts_quantize_rows(0, 0, 0, "
                      "0, 0, 0, 0, 0, 0) == HIST_ERR_INVALID_ARG ? EXPERTS_BF16 : 1; }\n")
    libdir = os.path.dirname(hist.LIBRARY)
    exe = str(tmp_path / "c")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                    build.INCLUDE, "-I", "/opt/rocm/include", str(source), "-L", libdir,
                    "-lpca_hist", f"-Wl,-rpath,{libdir}", "-o", exe], check=True,
                   capture_output=True)
    assert subprocess.run([exe], timeout=60).returncode == 0


def test_no_device_is_unsupported_not_a_crash():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert experts._library().experts_group(P, 32, 100, 8, 256, P, P, P, P, None, 0,
                                            None) == UNSUPPORTED
    assert experts._library().experts_quantize_rows(P, 64, P, P, 64, 10, 64, 0,
                                                    None) == UNSUPPORTED


def test_tensors_of_the_host_are_refused():
    ids = torch.zeros(4, 2, dtype=torch.int32)
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    g = experts.Groups(torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                       torch.zeros(8, dtype=torch.int32), ids)
    w = torch.zeros(3, 8, 16, dtype=torch.bfloat16)
    for call in (lambda: experts.group_rows(ids, 3), lambda: experts.quantize_rows(x),
                 lambda: experts.matmul(x, w, g, gather=True),
                 lambda: experts.linear(x, w, g, gather=True),
                 lambda: experts.combine(x, g), lambda: experts.matmul_dx(x, w, g),
                 lambda: experts.matmul_dw(x, x, g)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("source", [s for s in build.SOURCES if s.startswith("experts_")])
def test_no_scratch_and_no_spills(source, tmp_path):
    hipcc = build.hipcc() if os.path.exists(build.hipcc()) else shutil.which("hipcc")
    if not hipcc:
        pytest.skip("ROCm compiler not available")
    err = subprocess.run(
        [hipcc, *build.HIPCC_FLAGS, "--cuda-device-only", "-c", "-I", build.INCLUDE, "-I",
         build.CSRC, os.path.join(build.CSRC, source), "-o", str(tmp_path / "dev.o"),
         "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True,
        check=True).stderr
    names = re.findall(r"Function Name: (\S+)", err)
    scratch = [int(v) for v in re.findall(r"ScratchSize \[[^\]]*\]: (\d+)", err)]
    spills = [int(v) for v in re.findall(r"VGPRs Spill: (\d+)", err)]
    assert names and len(scratch) == len(spills) == len(names)
    bad = [r for r in zip(names, scratch, spills) if r[1] or r[2]]
    assert not bad, bad
