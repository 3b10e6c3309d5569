"""The shapes of tests/attn_forms.py reach every instance of the attention's
kernels that the library holds, by the launch plan itself (compiled from its
header): a bound of the plan that moves cannot leave an instance untested, and
an instance that no call reaches is found."""
import os
import re
import shutil
import subprocess

import pytest

import attn_forms

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "conv_subsampling_amd", "libdwconv.so")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not (shutil.which("g++") and shutil.which("nm")):
        pytest.skip("g++ or nm not found")
    exe = str(tmp_path_factory.mktemp("forms") / "attn_forms")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "conv_subsampling_amd", "csrc"), "-o", exe,
                    os.path.join(ROOT, "tests", "c", "attn_forms.cpp")], check=True)

    def forms(cases):
        out = subprocess.run([exe], input="\n".join(map(attn_forms.line, cases)) + "\n", capture_output=True, text=True,
                             check=True).stdout
        rows = [row.strip(";").split(";") for row in out.splitlines()]
        assert len(rows) == len(cases)
        return rows

    return forms


def held(kernel):
    syms = subprocess.run(["nm", "-C", LIB], capture_output=True, text=True, check=True).stdout
    return set(re.findall(rf"(?<=dw::){kernel}<[^>]*>", syms))


def test_every_instance_is_reached(plan):
    both, few = plan(attn_forms.self_attention()), plan(attn_forms.few_queries())
    assert {r[0] for r in both} | {r[0] for r in few} == held("attn_fwd_kernel")
    assert {r[1] for r in both} == held("attn_dq_kernel")
    assert {r[2] for r in both} == held("attn_dkv_kernel")


def test_shapes_own_the_frames_they_are_listed_for(plan):
    """float's widest heads own more where LDS asks for it."""
    cases = attn_forms.self_attention()
    for c, row in zip(cases, plan(cases)):
        own = [int(r.split(",")[2]) for r in row]
        assert own[0] == c["own"], (c, row)
        assert own[1] == c["own"] or (c["elem"] == 4 and c["D"] > 64 and own[1] > c["own"]), (c, row)
        assert own[2] == c["own"], (c, row)
