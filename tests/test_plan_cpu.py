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


# name: (the largest of the sums that the product's and the gradient's workspaces hold, M, N, K, adapters, rank)
WORKSPACES = {
    "few rows": (None, "out", 5, 4096, 4096, 3, 16),
    "few rows, many adapters": (None, "out", 16, 11008, 4096, 32, 72),
    "parts of K": ("out", "joined", 200, 2056, 5888, 3, 72),
    "parts of K and N": ("out", "out", 130, 1032, 1024, 2, 8),
    "parts of h": ("joined", "joined", 2048, 4096, 2048, 8, 32),
    "parts of h and the rows": ("joined", "grads", 4096, 4096, 4096, 1, 64),
    "parts of the rows": (None, "grads", 5000, 256, 512, 1, 64),
    "no parts": (None, None, 20000, 64, 64, 300, 8),
}


@pytest.mark.parametrize("name", list(WORKSPACES))
def test_workspace_bytes_are_those_of_the_parts(ask, name):
    """h (and u): their parts in binary32 for few rows, else three 16-bit numbers a value; behind them the sums that are
    joined, of which one kind at a time is needed."""
    forward, backward, M, N, K, adapters, rank = WORKSPACES[name]
    got = ask(("lora", M, N, K, adapters, rank))[0]
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for bwd, largest, (down, out, splits) in ((0, forward, (int(got[2]), int(got[3]), 1)),
                                            (1, backward, tuple(int(v) for v in got[4:]))):
        kinds, split = 1 + bwd, bwd or M > 96
        low = kinds * up(6 * M * rank if split else 4 * down * M * rank)
        sums = {"joined": up(4 * kinds * down * M * rank) if split and down > 1 else 0,
                "grads": up(4 * splits * adapters * rank * (N + K)) if splits > 1 else 0,
                "out": up(4 * out * M * (K if bwd else (N + 3) // 4 * 4)) if out > 1 else 0}
        assert (max(sums, key=sums.get) if any(sums.values()) else None) == largest
        assert q4.lib().q4_lora_workspace_bytes(M, N, K, adapters, rank, bwd) == low + max(sums.values())
