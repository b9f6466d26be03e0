"""The cache's operators used together: the example layer, a whole step captured
in a graph, and calls on another stream."""

import importlib.util
import os

import pytest
import torch

from bit_group_wise_amd import kv, q4
from _kv import DEV, Pool

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# A 4-bit value over groups of 32 is off by about a tenth of the group's spread
# (the step of 1/15 of the range, uniform), softmax weights follow the keys'
# error; the layer's output stays within a fifth of the 16-bit one's.
@pytest.mark.parametrize("fmt,g", [(q4.INT4_ASYM, 32), (q4.INT4_SYM, 32), (q4.NF4, 64)])
def test_example_layer(fmt, g):
    r = example().run(seqs=3, steps=70, budget=96, recent=16, fmt=fmt, g=g)
    assert r["prompt_difference"] < 0.2 and r["step_difference"] < 0.2, r
    assert r["evictions"] > 0
    assert r["device_lens"].tolist() == r["lens"]
    # every row's weights sum to one: what a token drew is never negative
    assert bool((r["mass"] >= 0).all()) and float(r["mass"].sum()) > 0


def test_step_in_a_graph():
    """append, attention with mass, read and evict captured once and replayed on
    changing inputs and lengths, each replay against the same calls made eagerly."""
    pool = Pool(q4.INT4_ASYM, 32, 128, 2, 16, [100, 60, 33], seed=4, spare=3 * 5)
    cache, table = pool.cache, pool.dev_table()
    free = [p for p in range(cache.pages) if p not in set(pool.table.reshape(-1).tolist())]
    new_table = torch.tensor(free[:15], dtype=torch.int32, device=DEV).view(3, 5)
    lens = torch.tensor([100, 60, 33], dtype=torch.int32, device=DEV)
    step = kv.Batch(table, lens)
    after_lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=DEV)
    after = kv.Batch(new_table, after_lens, starts, tokens=60, max_new=20)
    k, v = (torch.zeros((3, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device=DEV)
    mass = torch.zeros((3, 2, 112), device=DEV)

    def calls():
        kv.append(cache, step, k, v)
        out = kv.attention(cache, step, q, mass=mass)
        nl, nm, kept = kv.evict(cache, step, mass, new_table, 70, 9)
        after_lens.copy_(nl)
        return (out, nl, nm, kept, *kv.read(cache, after, torch.float16))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = calls()
    gen = torch.Generator(device=DEV)
    for i, n in enumerate(([100, 60, 33], [71, 70, 1], [99, 2, 33], [90, 60, 20])):
        gen.manual_seed(i)
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        mass.copy_(torch.rand(mass.shape, generator=gen, device=DEV))
        m0 = mass.clone()
        g.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in (*got, mass)]
        mass.copy_(m0)
        for a, b in zip(first, (*calls(), mass)):
            assert torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8)), i
        torch.cuda.synchronize()


def test_another_stream():
    """Calls run in order on the stream that is current, not on the tensors' first one."""
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 32, [64, 50], seed=4)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x = torch.randn((2, 2, 128), generator=gen, device=DEV).bfloat16()
    q = torch.randn((2, 4, 128), generator=gen, device=DEV).bfloat16()
    step = pool.batch()
    kv.append(pool.cache, step, x, x)
    want = kv.attention(pool.cache, step, q)
    kv.append(pool.cache, step, -x, -x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        kv.append(pool.cache, step, x, x)
        got = kv.attention(pool.cache, step, q)
    side.synchronize()
    assert torch.equal(got, want)
