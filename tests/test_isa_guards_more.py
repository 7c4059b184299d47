"""The build-time checks of test_isa_guards.py on the sources of the operators beside KDA: no
legacy bf16 matrix instruction, no matrix result read early, no packed fp32 arithmetic,
matrix cores where the work is theirs, and no kernel that uses scratch."""
import os
import re
import subprocess

import pytest

from chunked_gated_delta_12_amd import build as kbuild
from test_isa_guards import CSRC, _early_reads, _scratch_per_function

MATRIX = {"kda_gdr_prep.hip", "kda_gdr_chain.hip", "kda_gdr_grad.hip"}


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    try:
        hipcc = kbuild.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    tmp = tmp_path_factory.mktemp("isa")
    jobs = {}
    for src in kbuild.MORE_SOURCES:
        cmd = [hipcc] + kbuild._flags() + ["--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", str(tmp / (src + ".s")),
                                           "-Rpass-analysis=kernel-resource-usage"]
        jobs[src] = subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True)
    out = {}
    for src, p in jobs.items():
        err = p.communicate()[1]
        assert p.returncode == 0, err
        out[src] = ((tmp / (src + ".s")).read_text(), err)
    return out


@pytest.mark.parametrize("src", kbuild.MORE_SOURCES)
def test_instructions(assembly, src):
    text, _ = assembly[src]
    assert not re.findall(r"^\s*v_mfma_f32_16x16x16_?bf16", text, flags=re.M)
    assert not re.findall(r"^\s*v_pk_(?:add|mul|fma)_f32", text, flags=re.M)
    n = len(re.findall(r"^\s*v_mfma_f32_16x16x32_bf16", text, flags=re.M))
    assert (n > 0) == (src in MATRIX)


@pytest.mark.parametrize("src", kbuild.MORE_SOURCES)
def test_matrix_results_not_read_early(assembly, src):
    bad = _early_reads(assembly[src][0])
    assert not bad, f"{src}: matrix-core results read too early: {bad[:4]}"


# norm_bwd at 1,024 lanes a row keeps one or two kernel arguments in scratch, outside its loop.
_SCRATCH_ALLOWED = re.compile(r".*norm_bwd_kernelI(f|DF16b)Li1024E")


@pytest.mark.parametrize("src", kbuild.MORE_SOURCES)
def test_no_scratch(assembly, src):
    per = _scratch_per_function(assembly[src][1])
    bad = {fn: n for fn, n in per.items() if n and not (_SCRATCH_ALLOWED.match(fn) and n <= 16)}
    assert not bad, f"{src}: scratch use (bytes/lane): {bad}"
