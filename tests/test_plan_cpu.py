"""What sizes choose (csrc/plan.hpp, compiled for the host): the sizes of the GPU
tests reach the kernels that they are there for, and a workspace's bytes are
those that its parts need."""

import os
import shutil
import subprocess

import pytest

from bit_group_wise_amd import q4
from _sizes import EXPERTS, EXPERTS_DX, LORA, LORA_DX

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_group_wise_amd", "csrc")
GXX = shutil.which("g++") or shutil.which("c++")
pytestmark = pytest.mark.skipif(GXX is None, reason="needs g++")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    subprocess.run([GXX, "-std=c++20", "-O1", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "native", "plan.cpp"),
                    "-o", exe], check=True)

    def ask(*queries):
        out = subprocess.run([exe], input="\n".join(" ".join(map(str, q)) for q in queries), capture_output=True,
                             text=True, timeout=60, check=True).stdout
        return [line.split() for line in out.splitlines()]

    return ask


def test_experts_sizes(ask):
    got = ask(*(("experts", before + sum(counts) + behind, len(counts), N, K)
                for _, counts, before, behind, N, K, _ in EXPERTS.values()))
    assert [g[0] for g in got] == [v[0] for v in EXPERTS.values()]
    assert {v[0] for v in EXPERTS.values()} == {"stream1", "stream2", "skinny", "tile64", "tile128", "tile256"}


def test_experts_stream_sizes_give_a_workgroup_several_blocks():
    """Of 16 weight rows: more than are in flight (3) and than one join of sums takes (4)."""
    most = {}
    for kernel, counts, _, _, N, K, _ in EXPERTS.values():
        if kernel.startswith("stream"):
            rows = 16 if kernel == "stream1" else 32
            blocks = sum((n + rows - 1) // rows for n in counts) * ((N + 15) // 16)
            key = kernel, K > 2048
            most[key] = max(most.get(key, 0), blocks / 256)
    assert len(most) == 4 and min(most.values()) > 6


def test_experts_gradient_sizes(ask):
    got = ask(*(("experts", before + sum(counts) + behind, len(counts), N, K)
                for _, counts, before, behind, N, K, _ in EXPERTS_DX.values()))
    assert [int(g[1]) for g in got] == [v[0] for v in EXPERTS_DX.values()]
    quarters = {(n % 256 + 63) // 64 for v in EXPERTS_DX.values() if v[0] == 256 for n in v[1]}
    assert {1, 2, 3, 4} <= quarters


def test_lora_sizes(ask):
    got = ask(*(("lora", M, N, K, 3, 16) for _, M, N, K, _ in LORA.values()))
    assert [g[0] for g in got] == [v[0] for v in LORA.values()]
    assert {v[0] for v in LORA.values()} == {"skinny", "tile64", "tile128", "tile256"}
    assert {int(g[3]) > 1 for g in got if g[0] == "tile64"} == {True, False}


def test_lora_gradient_sizes(ask):
    got = ask(*(("lora", M, N, K, 3, 16) for _, _, M, N, K, _ in LORA_DX.values()))
    assert [(int(g[1]), int(g[5])) for g in got] == [v[:2] for v in LORA_DX.values()]
