"""Products through experts' weights (q4_experts_*) against binary64 products
with the dequantized weights, expert by expert: every kernel that the mean
number of rows can choose, all formats, ragged and empty groups, gathered
rows, sizes that fill no tile, and what lies outside the groups."""

import pytest
import torch

from bit_group_wise_amd import experts, q4
from _groups import ACTS, DEV, FORMATS, assert_product, generator, normal, values, weight
from _sizes import EXPERTS, EXPERTS_DX

pytestmark = pytest.mark.gpu


def offsets_of(counts, first=0):
    o = [first]
    for n in counts:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device=DEV)


def groups(offsets):
    o = offsets.tolist()
    return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(o, o[1:])) if hi > lo]


def check(x, q, offsets, index=None, out=None, tag=""):
    """experts.gemm against the definition; returns its output."""
    act = q4.F16 if x.dtype == torch.float16 else q4.BF16
    N = q.N // (offsets.numel() - 1)
    y = experts.gemm(x, q, offsets, index=index, out=out)
    w = values(q, act)
    for e, lo, hi in groups(offsets):
        rows = x[lo:hi] if index is None else x[index[lo:hi].long().clamp(0, x.shape[0] - 1)]
        rows = rows.double()
        if index is not None:
            rows = rows * ((index[lo:hi] >= 0) & (index[lo:hi] < x.shape[0]))[:, None]
        we = w[e * N:(e + 1) * N]
        assert_product(y[lo:hi], rows @ we.T, rows.abs() @ we.abs().T, q.K, act, f"{tag} expert {e}")
    return y


def check_dx(dy, q, offsets, out=None, tag=""):
    act = q4.F16 if dy.dtype == torch.float16 else q4.BF16
    N = dy.shape[1]
    dx = experts.gemm_dx(dy, q, offsets, out=out)
    w = values(q, act)
    for e, lo, hi in groups(offsets):
        we = w[e * N:(e + 1) * N]
        d = dy[lo:hi].double()
        assert_product(dx[lo:hi], d @ we, d.abs() @ we.abs(), N, act, f"{tag} expert {e}")
    return dx


# small groups: streamed, and in tiles of 64 rows (sizes that reach each kernel: EXPERTS below)
COUNTS = {
    "one": [0, 1, 0, 0],
    "few": [3, 0, 17, 5, 1],
    "some": [20, 31, 0, 40, 16],
    "tens": [64, 33, 0, 70],
    "hundred": [128, 1, 200, 130],
    "hundreds": [300, 0, 513, 256],
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("fmt", FORMATS)
def test_groups_of_any_size(fmt, name):
    counts = COUNTS[name]
    act, g = (q4.BF16, 64) if FORMATS.index(fmt) % 2 else (q4.F16, 32)
    gen = generator(7 * fmt + len(name))
    N, K = 144, 448 if g == 64 else 352
    q = weight(len(counts) * N, K, fmt, g, gen)
    x = normal(gen, act, sum(counts), K)
    check(x, q, offsets_of(counts))
    check_dx(normal(gen, act, sum(counts), N), q, offsets_of(counts))


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_one_expert(rows):
    gen = generator(rows)
    q = weight(264, 256, q4.INT4_ASYM, 32, gen)
    check(normal(gen, q4.BF16, rows, 256), q, offsets_of([rows]))
    check_dx(normal(gen, q4.F16, rows, 264), q, offsets_of([rows]))


@pytest.mark.parametrize("N,K,g", [(1, 32, 32), (79, 96, 32), (15, 128, 128), (257, 192, 64), (130, 1120, 32),
                                   (33, 4096, 128)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_odd_weights(fmt, N, K, g):
    """Weights whose rows fill no block: an expert's zero-points may start in the middle of a byte, its constants in the middle of a run."""
    gen = generator(N + K)
    for counts in ([2, 0, 1], [70, 3, 40], [150, 200, 131]):
        q = weight(3 * N, K, fmt, g, gen)
        check(normal(gen, q4.BF16, sum(counts), K), q, offsets_of(counts))
        if N % 8 == 0:
            check_dx(normal(gen, q4.BF16, sum(counts), N), q, offsets_of(counts))


@pytest.mark.parametrize("N,K,g", [(8, 32, 32), (72, 96, 32), (136, 192, 64), (264, 384, 128)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_odd_gradients(fmt, N, K, g):
    gen = generator(N + K)
    for counts in ([2, 0, 1], [150, 200, 131]):
        q = weight(3 * N, K, fmt, g, gen)
        check_dx(normal(gen, q4.F16, sum(counts), N), q, offsets_of(counts))


@pytest.mark.parametrize("experts_", [64, 65, 130, 300])
def test_many_experts(experts_):
    gen = generator(experts_)
    counts = torch.randint(0, 6, (experts_,), generator=gen, device=DEV).tolist()
    counts[experts_ // 2] = 40  # one that takes several pieces
    q = weight(experts_ * 16, 64, q4.INT4_SYM, 32, gen)
    check(normal(gen, q4.BF16, sum(counts), 64), q, offsets_of(counts))
    check_dx(normal(gen, q4.BF16, sum(counts), 16), q, offsets_of(counts))


@pytest.mark.parametrize("counts", [[3, 0, 9], [60, 35, 41], [190, 257, 300]])
@pytest.mark.parametrize("K", [64, 160, 4096])
def test_gathered_rows(counts, K):
    gen = generator(sum(counts) + K)
    rows, tokens, N = sum(counts), 11 + sum(counts) // 3, 96
    q = weight(3 * N, K, q4.NF4, 32, gen)
    x = normal(gen, q4.F16, tokens, K)
    index = torch.randint(0, tokens, (rows,), generator=gen, device=DEV).int()
    y = check(x, q, offsets_of(counts), index)
    # gathering first gives the same bits
    assert torch.equal(y, experts.gemm(x[index.long()], q, offsets_of(counts)))
    # indexes outside x: rows of zeros
    index[::5], index[1::7] = -1, tokens
    index[2::11] = 2 ** 31 - 1
    y = check(x, q, offsets_of(counts), index)
    out = (index < 0) | (index >= tokens)
    assert bool((y[out] == 0).all())


@pytest.mark.parametrize("counts", [[4, 0, 9], [60, 35, 41], [190, 257, 300]])
@pytest.mark.parametrize("K,N", [(96, 72), (256, 64), (1120, 136)])
def test_rows_outside_the_groups(counts, K, N):
    """Rows before the first group and behind the last hold NaN, stay as they were and reach no other row."""
    gen = generator(sum(counts) + K)
    before, behind, n = 5, 130, sum(counts)
    q = weight(3 * N, K, q4.INT4_ASYM, 32, gen)
    off = offsets_of(counts, before)
    for width, call in ((K, check), (N, check_dx)):
        x = normal(gen, q4.BF16, before + n + behind, width)
        x[:before], x[before + n:] = float("nan"), float("inf")
        y = torch.full((x.shape[0], N + K - width), 3.0, dtype=x.dtype, device=DEV)
        call(x, q, off, out=y)
        assert bool((y[:before] == 3).all()) and bool((y[before + n:] == 3).all())


@pytest.mark.parametrize("counts", [[2, 3, 2], [40, 70, 61], [200, 290, 180]])
@pytest.mark.parametrize("K,N", [(96, 72), (512, 64)])
def test_a_row_that_is_not_finite_reaches_its_own_output_alone(counts, K, N):
    gen = generator(K + sum(counts))
    q = weight(3 * N, K, q4.NF4, 32, gen)
    off = offsets_of(counts)
    bad = counts[0] + counts[1] // 2
    for width, call in ((K, experts.gemm), (N, experts.gemm_dx)):
        x = normal(gen, q4.F16, sum(counts), width)
        clean = call(x, q, off)
        x[bad] = float("nan")
        y = call(x, q, off)
        assert bool(torch.isnan(y[bad]).all())
        keep = torch.arange(x.shape[0], device=DEV) != bad
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("offs", [[0, 9, 4, 20], [7, 3, 12, 20], [-5, 8, 8, 1 << 30], [20, 0, 0, 0],
                                  [0, 0, 0, 0], [-9, -8, -7, -1], [0, -2 ** 31, 2 ** 31 - 1, 5]])
def test_offsets_that_are_none(offs):
    """Offsets are held to the rows, one below an earlier one counts as that: nothing else is written."""
    gen = generator(3)
    N, K, rows = 40, 64, 20
    q = weight(3 * N, K, q4.INT4_SYM, 32, gen)
    x, dy = normal(gen, q4.BF16, rows, K), normal(gen, q4.BF16, rows, N)
    high, clean = 0, []
    for o in offs:
        high = max(high, min(max(o, 0), rows))
        clean.append(high)
    clean = torch.tensor(clean, dtype=torch.int32, device=DEV)
    offs = torch.tensor(offs, dtype=torch.int32, device=DEV)
    for call, arg, width in ((experts.gemm, x, N), (experts.gemm_dx, dy, K)):
        got = torch.full((rows, width), 3.0, dtype=x.dtype, device=DEV)
        want = got.clone()
        call(arg, q, offs, out=got)
        call(arg, q, clean, out=want)
        assert torch.equal(got, want)


def test_no_rows():
    gen = generator(1)
    q = weight(4 * 64, 64, q4.NF4, 64, gen)
    off = offsets_of([0, 0, 0, 0])
    x = normal(gen, q4.BF16, 3, 64)
    assert experts.gemm(x[:0], q, off).shape == (0, 64)
    assert experts.gemm(x, q, off, index=off[:0]).shape == (0, 64)
    assert experts.gemm_dx(x[:0], q, off).shape == (0, 64)


def test_order_of_calls_and_choice_give_close_results():
    """The same rows in one group of many and in groups that choose other kernels."""
    gen = generator(5)
    N, K = 256, 512
    one = weight(N, K, q4.INT4_SYM, 64, gen)
    x = normal(gen, q4.BF16, 600, K)
    big = check(x, one, offsets_of([600]))
    small = torch.cat([check(x[i:i + 12], one, offsets_of([12])) for i in range(0, 600, 12)])
    assert float((big.double() - small.double()).abs().max()) <= 2.0 ** -7 * float(big.abs().max())


def test_captured_and_replayed_with_other_groups():
    gen = generator(9)
    N, K, rows = 96, 128, 64
    q = weight(4 * N, K, q4.NF4, 64, gen)
    x, dy = normal(gen, q4.BF16, rows, K), normal(gen, q4.BF16, rows, N)
    off = offsets_of([16, 16, 16, 16])
    y, dx = torch.zeros((rows, N), dtype=x.dtype, device=DEV), torch.zeros((rows, K), dtype=x.dtype, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        experts.gemm(x, q, off, out=y)
        experts.gemm_dx(dy, q, off, out=dx)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        experts.gemm(x, q, off, out=y)
        experts.gemm_dx(dy, q, off, out=dx)
    for counts in ([64, 0, 0, 0], [0, 1, 62, 1], [13, 20, 0, 31], [0, 0, 0, 64]):
        off.copy_(offsets_of(counts))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, experts.gemm(x, q, off)) and torch.equal(dx, experts.gemm_dx(dy, q, off))


def test_outputs_at_any_two_bytes():
    """y may start at any element; its neighbours stay."""
    gen = generator(4)
    N, K = 72, 64
    for counts in ([5, 6], [50, 40], [300, 200]):
        q = weight(2 * N, K, q4.INT4_SYM, 32, gen)
        x = normal(gen, q4.BF16, sum(counts), K)
        flat = torch.full((sum(counts) * N + 8,), 3.0, dtype=x.dtype, device=DEV)
        y = flat[3:3 + sum(counts) * N].view(-1, N)
        check(x, q, offsets_of(counts), out=y)
        assert bool((flat[:3] == 3).all()) and bool((flat[3 + sum(counts) * N:] == 3).all())


def test_arguments():
    gen = generator(2)
    q = weight(3 * 64, 64, q4.NF4, 64, gen)
    x, off = normal(gen, q4.BF16, 6, 64), offsets_of([1, 2, 3])
    with pytest.raises(ValueError):
        experts.gemm(x[:, :32], q, off)
    with pytest.raises(ValueError):
        experts.gemm(x, q, offsets_of([1, 1, 1, 1, 2]))  # 192 rows are not five experts'
    with pytest.raises(TypeError):
        experts.gemm(x, q, off.long())
    with pytest.raises(TypeError):
        experts.gemm(x.float(), q, off)
    with pytest.raises(ValueError):
        experts.gemm(x.cpu(), q, off)
    with pytest.raises(ValueError):
        experts.gemm(x, q, off, out=x.new_empty((5, 64)))
    with pytest.raises(ValueError):
        experts.gemm_dx(x[:, :32].contiguous(), q, off)
    with pytest.raises(TypeError):
        experts.gemm(x, q, off, index=off[:3].float())


def framed(act, rows, width, before, behind, value):
    """[before + rows + behind, width] of `value`, beginning at an odd element, and its flat storage."""
    n = (before + rows + behind) * width
    flat = torch.full((n + 16,), value, dtype=ACTS[act], device=DEV)
    return flat[1:1 + n].view(-1, width), flat


def kept(y, flat, before, rows, value):
    """Whether all but the groups' rows still holds `value`."""
    y = y.clone()
    inside = y[before:before + rows].numel()
    return (int((flat == value).sum()) - int((y[before:before + rows] == value).sum())) == flat.numel() - inside


@pytest.mark.parametrize("name", list(EXPERTS))
@pytest.mark.parametrize("fmt", FORMATS)
def test_each_kernel(fmt, name):
    """Rows as they lie, gathered ones, bad indexes, rows outside the groups, a row of NaN, outputs at any element."""
    _, counts, before, behind, N, K, g = EXPERTS[name]
    gen = generator(fmt + N + K)
    n, act = sum(counts), (fmt + len(name)) % 2
    q = weight(len(counts) * N, K, fmt, g, gen)
    off = offsets_of(counts, before)
    x = normal(gen, act, before + n + behind, K)
    x[:before], x[before + n:] = float("nan"), float("inf")
    y = torch.full((before + n + behind, N), 3.0, dtype=x.dtype, device=DEV)
    check(x, q, off, out=y, tag=name)
    assert bool((y[:before] == 3).all()) and bool((y[before + n:] == 3).all())

    bad = before + n // 2
    x[bad] = float("nan")
    again = experts.gemm(x, q, off)
    assert bool(torch.isnan(again[bad]).all())
    inside = torch.arange(x.shape[0], device=DEV)
    inside = (inside >= before) & (inside < before + n) & (inside != bad)
    assert torch.equal(again[inside], y[inside])

    tokens = 3 + n // 2
    t = normal(gen, act, tokens, K)
    index = torch.randint(0, tokens, (x.shape[0],), generator=gen, device=DEV).int()
    index[:before], index[before + n:] = tokens, -7
    index[before:before + n][::5], index[before:before + n][3::7] = -1, tokens
    got, flat = framed(act, n, N, before, behind, 3.0)
    got = check(t, q, off, index, out=got, tag=f"{name} gathered")
    none = (index < 0) | (index >= tokens)
    none[:before], none[before + n:] = False, False
    assert bool((got[none] == 0).all()) and kept(got, flat, before, n, 3.0)


@pytest.mark.parametrize("name", list(EXPERTS_DX))
@pytest.mark.parametrize("fmt", FORMATS)
def test_each_gradient_kernel(fmt, name):
    _, counts, before, behind, N, K, g = EXPERTS_DX[name]
    gen = generator(fmt + N + K)
    n, act = sum(counts), (fmt + len(name)) % 2
    q = weight(len(counts) * N, K, fmt, g, gen)
    off = offsets_of(counts, before)
    dy = normal(gen, act, before + n + behind, N)
    dy[:before], dy[before + n:] = float("nan"), float("inf")
    dx = torch.full((before + n + behind, K), 3.0, dtype=dy.dtype, device=DEV)
    check_dx(dy, q, off, out=dx, tag=name)
    assert bool((dx[:before] == 3).all()) and bool((dx[before + n:] == 3).all())
    bad = before + n // 2
    dy[bad] = float("nan")
    again = experts.gemm_dx(dy, q, off)
    assert bool(torch.isnan(again[bad]).all())
    inside = torch.arange(dy.shape[0], device=DEV)
    inside = (inside >= before) & (inside < before + n) & (inside != bad)
    assert torch.equal(again[inside], dx[inside])


@pytest.mark.parametrize("name", ["stream1", "stream2", "skinny", "tile128", "tile256"])
def test_each_kernel_captured_and_replayed_with_other_groups(name):
    _, counts, before, behind, N, K, g = EXPERTS[name]
    gen = generator(N)
    rows = before + sum(counts) + behind
    q = weight(len(counts) * N, K, q4.NF4_DQ, g, gen)
    x, off = normal(gen, q4.BF16, rows, K), offsets_of(counts, before)
    y = torch.zeros((rows, N), dtype=x.dtype, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        experts.gemm(x, q, off, out=y)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        experts.gemm(x, q, off, out=y)
    for k in range(4):
        cuts = torch.randint(0, rows + 1, (len(counts) + 1,), generator=gen, device=DEV).sort().values.int()
        off.copy_(cuts if k < 3 else torch.full_like(cuts, rows).index_fill_(0, torch.tensor([0], device=DEV), 0))
        y.zero_()
        x.copy_(normal(gen, q4.BF16, rows, K))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(y)
        check(x, q, off, out=want, tag=f"{name} {k}")
        assert torch.equal(y, want)
