"""Low-rank adapters beside a 4-bit weight (q4_lora_*) against the formulas in
binary64: every kernel, rank and mixture of adapters, gradients also against
differences, and what an adapter or a row that is not finite may reach."""

import ctypes

import pytest
import torch

from bit_group_wise_amd import lora, q4
from _groups import ACTS, DEV, FORMATS, generator, half_step, normal, tiny, values, weight
from _sizes import LORA, LORA_DX

pytestmark = pytest.mark.gpu


def pairs_of(gen, act, adapters, rank, N, K, scale=True, size=1.0):
    s = (torch.rand((adapters,), generator=gen, device=DEV) + 0.5) if scale else None
    return lora.Adapters(normal(gen, act, adapters, rank, K, size=size * K ** -0.5),
                         normal(gen, act, adapters, N, rank, size=rank ** -0.5), s)


def ids_of(gen, M, adapters, kind):
    if kind == "none":
        return None
    if kind == "runs":  # sorted, some rows with none
        return (torch.arange(M, device=DEV) * (adapters + 1) // max(M, 1) - 1).int()
    ids = torch.randint(-1, adapters + 1, (M,), generator=gen, device=DEV).int()  # -1 and `adapters`: none
    if M > 3:
        ids[M // 3], ids[M // 2] = 2 ** 31 - 1, -2 ** 31
    return ids


def of_rows(pairs, ids, M):
    """[(adapter, its rows, its scale)] and matrices in binary64."""
    ids = torch.zeros((M,), device=DEV) if ids is None else ids
    scale = torch.ones((pairs.adapters,), device=DEV) if pairs.scale is None else pairs.scale
    return [(i, (ids == i).nonzero()[:, 0], float(scale[i].double())) for i in range(pairs.adapters)]


def assert_within(got, want, sums, act, tag):
    """The sum's error, and the rounding of what it makes."""
    assert bool(torch.isfinite(got).all()), f"{tag} not finite"
    worst = ((got.double() - want).abs() - (sums + half_step(act) * (want.abs() + sums) + tiny(act))).max()
    assert bool(worst <= 0), f"{tag} past the tolerance by {float(worst)}"


# Errors relative to the sums of magnitudes: an addition in binary32 at most
# 2^-23 (the matrix cores may cut where they do not round).  TWO_PARTS is room
# for h and u as two bfloat16 numbers, 2^-18 (2^-9 of 2^-9), and fp16's product
# of second parts, 2^-18; that they enter with all their bits is tested by whole
# numbers (test_every_bit_of_the_low_product and its gradients).
def short(terms):
    return terms * 2.0 ** -23


TWO_PARTS = 2.0 ** -17


def check(x, q, pairs, ids, tag="", **kw):
    act = q4.F16 if x.dtype == torch.float16 else q4.BF16
    M, K, R = x.shape[0], pairs.K, pairs.rank
    y = lora.gemm(x, q, pairs, ids, **kw)
    w, xd = values(q, act), x.double()
    want, sums = xd @ w.T, short(K + 1) * (xd.abs() @ w.abs().T)
    for i, rows, s in of_rows(pairs, ids, M):
        a, b = pairs.a[i].double(), pairs.b[i].double()
        want[rows] += s * (xd[rows] @ a.T) @ b.T
        low = s * (xd[rows].abs() @ a.abs().T) @ b.abs().T
        sums[rows] += low * (short(K + 16 + 3 * R) + TWO_PARTS)
    assert_within(y, want, sums, act, tag)
    return y


def check_backward(dy, x, q, pairs, ids, tag="", **kw):
    act = q4.F16 if x.dtype == torch.float16 else q4.BF16
    M, N, K, R = x.shape[0], pairs.N, pairs.K, pairs.rank
    dx, da, db = lora.backward(dy, x, q, pairs, ids, **kw)
    w, xd, d = values(q, act), x.double(), dy.double()
    want, sums = d @ w, short(N + 1) * (d.abs() @ w.abs())
    for i, rows, s in of_rows(pairs, ids, M):
        a, b, xr, dr = pairs.a[i].double(), pairs.b[i].double(), xd[rows], d[rows]
        u, ub = s * dr @ b, s * dr.abs() @ b.abs()
        h, hb = s * xr @ a.T, s * xr.abs() @ a.abs().T
        want[rows] += u @ a
        sums[rows] += (ub @ a.abs()) * (short(N + 16 + 3 * R) + TWO_PARTS)
        many = 3 * len(rows) + 16
        assert_within(da[i], u.T @ xr, (ub.T @ xr.abs()) * (short(N + many) + TWO_PARTS), act, f"{tag} da {i}")
        assert_within(db[i], dr.T @ h, (dr.abs().T @ hb) * (short(K + many) + TWO_PARTS), act, f"{tag} db {i}")
    assert_within(dx, want, sums, act, f"{tag} dx")
    return dx, da, db


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 65, 97, 256, 513])
@pytest.mark.parametrize("kind,adapters,rank", [("none", 1, 16), ("runs", 3, 8), ("mixed", 5, 40), ("mixed", 70, 64)])
def test_rows(M, kind, adapters, rank):
    gen = generator(M + rank)
    fmt, act = FORMATS[(M + rank) % 5], (M + rank) // 8 % 2
    q = weight(144, 320, fmt, 32, gen)
    pairs = pairs_of(gen, act, adapters, rank, 144, 320)
    ids = ids_of(gen, M, adapters, kind)
    x, dy = normal(gen, act, M, 320), normal(gen, act, M, 144)
    check(x, q, pairs, ids)
    check_backward(dy, x, q, pairs, ids)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 48, 64, 72, 128, 200, 256])
@pytest.mark.parametrize("M", [5, 70, 150])
@pytest.mark.parametrize("act", [q4.F16, q4.BF16])
def test_ranks(rank, M, act):
    gen = generator(rank + M)
    q = weight(80, 256, q4.NF4, 64, gen)
    pairs = pairs_of(gen, act, 3, rank, 80, 256)
    ids = ids_of(gen, M, 3, "mixed")
    x, dy = normal(gen, act, M, 256), normal(gen, act, M, 80)
    check(x, q, pairs, ids)
    check_backward(dy, x, q, pairs, ids)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("act", [q4.F16, q4.BF16])
def test_formats(fmt, g, act):
    gen = generator(fmt * 7 + g)
    N, K = 264, 640
    q = weight(N, K, fmt, g, gen)
    pairs = pairs_of(gen, act, 2, 16, N, K)
    for M in (3, 30, 60, 200, 600):
        ids = ids_of(gen, M, 2, "runs")
        x, dy = normal(gen, act, M, K), normal(gen, act, M, N)
        check(x, q, pairs, ids, f"M {M}")
        if M in (3, 600):
            check_backward(dy, x, q, pairs, ids, f"M {M}")


@pytest.mark.parametrize("N,K", [(1, 32), (79, 96), (130, 1120), (257, 4096), (1000, 64)])
@pytest.mark.parametrize("M", [1, 40, 130, 520])
def test_odd_sizes(M, N, K):
    gen = generator(M + N + K)
    q = weight(N, K, q4.INT4_ASYM, 32, gen)
    pairs = pairs_of(gen, q4.BF16, 4, 24, N, K)
    ids = ids_of(gen, M, 4, "mixed")
    check(normal(gen, q4.BF16, M, K), q, pairs, ids)


@pytest.mark.parametrize("N,K", [(8, 32), (72, 96), (136, 1120), (264, 4096), (4096, 64)])
@pytest.mark.parametrize("M", [1, 40, 130, 1100])
def test_odd_gradients(M, N, K):
    gen = generator(M + N + K)
    q = weight(N, K, q4.INT4_ASYM, 32, gen)
    pairs = pairs_of(gen, q4.F16, 4, 24, N, K)
    ids = ids_of(gen, M, 4, "mixed")
    check_backward(normal(gen, q4.F16, M, N), normal(gen, q4.F16, M, K), q, pairs, ids)


@pytest.mark.parametrize("N,K", [(1, 1024), (130, 2272), (147, 5888), (256, 3328)])
@pytest.mark.parametrize("M", [97, 200, 450])
@pytest.mark.parametrize("fmt", FORMATS)
def test_long_rows(M, N, K, fmt):
    """K in parts on different workgroups, their sums joined; rows of no adapter among them."""
    gen = generator(M + N + K)
    q = weight(N, K, fmt, 32, gen)
    for act in (q4.F16, q4.BF16):
        pairs = pairs_of(gen, act, 3, 72, N, K)
        ids = ids_of(gen, M, 3, "mixed")
        check(normal(gen, act, M, K), q, pairs, ids)


@pytest.mark.parametrize("N,K", [(2048, 128), (4104, 96), (7640, 640)])
@pytest.mark.parametrize("M", [1, 70, 333])
@pytest.mark.parametrize("act", [q4.F16, q4.BF16])
def test_gradients_of_long_outputs(M, N, K, act):
    """N in parts on different workgroups, their sums joined; rows of no adapter among them."""
    gen = generator(M + N + K)
    q = weight(N, K, q4.NF4_DQ if K % 64 == 0 else q4.INT4_ASYM, 64 if K % 64 == 0 else 32, gen)
    pairs = pairs_of(gen, act, 3, 72, N, K)
    ids = ids_of(gen, M, 3, "mixed")
    check_backward(normal(gen, act, M, N), normal(gen, act, M, K), q, pairs, ids)


def test_many_rows_of_one_adapter():
    """Rows split over workgroups, their sums joined; no ids, no scale."""
    gen = generator(6)
    q = weight(256, 512, q4.NF4_DQ, 64, gen)
    for act in (q4.F16, q4.BF16):
        pairs = pairs_of(gen, act, 1, 64, 256, 512, scale=False)
        x, dy = normal(gen, act, 5000, 512), normal(gen, act, 5000, 256)
        check(x, q, pairs, None)
        check_backward(dy, x, q, pairs, None)


def test_every_row_its_own_adapter():
    gen = generator(8)
    M = 300
    q = weight(64, 128, q4.NF4, 64, gen)
    pairs = pairs_of(gen, q4.BF16, M, 8, 64, 128)
    ids = torch.randperm(M, generator=gen, device=DEV).int()
    x, dy = normal(gen, q4.BF16, M, 128), normal(gen, q4.BF16, M, 64)
    check(x, q, pairs, ids)
    check_backward(dy, x, q, pairs, ids)
    check(x[:64], q, pairs, ids[:64])


def test_many_rows_of_many_adapters():
    """More steps of rows than a workgroup lists at a time, most without a row of its adapter."""
    gen = generator(16)
    M, A = 20000, 300
    q = weight(64, 64, q4.NF4, 64, gen)
    pairs = pairs_of(gen, q4.BF16, A, 8, 64, 64)
    ids = torch.randint(-1, A, (M,), generator=gen, device=DEV).int()
    ids[:16500] = torch.where(ids[:16500] == 7, 8, ids[:16500])  # adapter 7: in the last steps alone
    check_backward(normal(gen, q4.BF16, M, 64), normal(gen, q4.BF16, M, 64), q, pairs, ids)


@pytest.mark.parametrize("M", [3, 64, 200, 600])
def test_rows_without_an_adapter_are_the_products_own(M):
    """The same bits as q4.gemm and q4.gemm_dx, and gradients of zero."""
    gen = generator(M)
    q = weight(128, 256, q4.INT4_SYM, 64, gen)
    pairs = pairs_of(gen, q4.BF16, 2, 16, 128, 256)
    ids = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    x, dy = normal(gen, q4.BF16, M, 256), normal(gen, q4.BF16, M, 128)
    assert torch.equal(lora.gemm(x, q, pairs, ids), q4.gemm(x, q))
    dx, da, db = lora.backward(dy, x, q, pairs, ids)
    assert torch.equal(dx, q4.gemm_dx(dy, q))
    assert not da.any() and not db.any()


@pytest.mark.parametrize("M", [20, 90, 300, 700])
@pytest.mark.parametrize("act", [q4.F16, q4.BF16])
def test_an_adapter_that_is_not_finite_reaches_its_own_rows_alone(M, act):
    gen = generator(M)
    q = weight(72, 96, q4.NF4, 32, gen)
    pairs = pairs_of(gen, act, 4, 24, 72, 96)
    ids = ids_of(gen, M, 4, "mixed")
    x, dy = normal(gen, act, M, 96), normal(gen, act, M, 72)
    clean, grads = lora.gemm(x, q, pairs, ids), lora.backward(dy, x, q, pairs, ids)
    for part, bad in (("a", float("nan")), ("b", float("inf")), ("scale", float("nan"))):
        new = lora.Adapters(pairs.a.clone(), pairs.b.clone(), pairs.scale.clone())
        getattr(new, part)[2] = bad
        others = ids != 2
        y, (dx, da, db) = lora.gemm(x, q, new, ids), lora.backward(dy, x, q, new, ids)
        assert torch.equal(y[others], clean[others]) and not torch.isfinite(y[~others]).all()
        assert torch.equal(dx[others], grads[0][others])
        for got, want in ((da, grads[1]), (db, grads[2])):
            assert torch.equal(got[[0, 1, 3]], want[[0, 1, 3]])


@pytest.mark.parametrize("M", [20, 90, 300, 700])
@pytest.mark.parametrize("N,K", [(72, 96), (128, 512)])
def test_a_row_that_is_not_finite_reaches_its_own_alone(M, N, K):
    gen = generator(M + K)
    q = weight(N, K, q4.INT4_ASYM, 32, gen)
    pairs = pairs_of(gen, q4.BF16, 3, 16, N, K)
    ids = ids_of(gen, M, 3, "mixed")
    bad = M // 2 + 1
    ids[bad] = 1
    x, dy = normal(gen, q4.BF16, M, K), normal(gen, q4.BF16, M, N)
    clean, grads = lora.gemm(x, q, pairs, ids), lora.backward(dy, x, q, pairs, ids)
    x[bad], dy[bad] = float("nan"), float("inf")
    keep = torch.arange(M, device=DEV) != bad
    y, (dx, da, db) = lora.gemm(x, q, pairs, ids), lora.backward(dy, x, q, pairs, ids)
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[bad]).all())
    assert torch.equal(dx[keep], grads[0][keep]) and not torch.isfinite(dx[bad]).any()
    for got, want in ((da, grads[1]), (db, grads[2])):
        assert torch.equal(got[[0, 2]], want[[0, 2]])


@pytest.mark.parametrize("M", [4, 100, 600])
def test_fp16_far_from_one(M):
    """h past fp16's range, and gradients below it, in fp16."""
    gen = generator(M)
    N, K = 96, 512
    q = weight(N, K, q4.NF4, 64, gen)
    a = normal(gen, q4.F16, 1, 16, K, size=40.0)
    x = normal(gen, q4.F16, M, K, size=100.0)
    b = normal(gen, q4.F16, 1, N, 16, size=1e-3)
    pairs = lora.Adapters(a, b)
    assert float((x.double() @ a[0].double().T).abs().max()) > 65504
    check(x, q, pairs, None)
    # u is about 2^-24 and smaller; its products are numbers again
    dy = normal(gen, q4.F16, M, N, size=1e-4)
    pairs = lora.Adapters(normal(gen, q4.F16, 1, 16, K, size=1000.0), normal(gen, q4.F16, 1, N, 16, size=1e-4))
    assert float((dy.double() @ pairs.b[0].double()).abs().max()) < 2.0 ** -17
    check_backward(dy, x, q, pairs, None)


def test_gradients_against_differences():
    """Along a direction, with y in binary64: what the gradients say up to their rounding."""
    gen = generator(11)
    M, N, K, R = 150, 64, 96, 16
    act = q4.BF16
    q = weight(N, K, q4.NF4, 32, gen)
    pairs = pairs_of(gen, act, 2, R, N, K)
    ids = ids_of(gen, M, 2, "mixed")
    x, dy = normal(gen, act, M, K), normal(gen, act, M, N)
    grads = lora.backward(dy, x, q, pairs, ids)
    w = values(q, act)

    def loss(x, a, b):
        y = x @ w.T
        for i, rows, s in of_rows(pairs, ids, M):
            y[rows] = y[rows] + s * (x[rows] @ a[i].T) @ b[i].T
        return float((y * dy.double()).sum())

    at = [x.double(), pairs.a.double(), pairs.b.double()]
    for k, g in enumerate(grads):
        way = torch.randn(at[k].shape, generator=gen, device=DEV, dtype=torch.float64)
        step = 1e-3
        ahead, behind = list(at), list(at)
        ahead[k], behind[k] = at[k] + step * way, at[k] - step * way
        rate = (loss(*ahead) - loss(*behind)) / (2 * step)  # (exact: the loss is linear in each)
        said, rough = float((g.double() * way).sum()), float((g.double() * way).abs().sum())
        assert abs(rate - said) <= rough * (half_step(act) + TWO_PARTS + short(M * 4)) + 1e-6 * rough


def test_parts_alone_and_again():
    """Each output alone, twice, into given tensors and from a workspace full of NaN: the same bits."""
    gen = generator(12)
    M, N, K = 700, 128, 256
    q = weight(N, K, q4.INT4_SYM, 64, gen)
    pairs = pairs_of(gen, q4.F16, 3, 40, N, K)
    ids = ids_of(gen, M, 3, "mixed")
    x, dy = normal(gen, q4.F16, M, K), normal(gen, q4.F16, M, N)
    y, (dx, da, db) = lora.gemm(x, q, pairs, ids), lora.backward(dy, x, q, pairs, ids)
    work = torch.full((lora.workspace_bytes(M, pairs, True),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(lora.gemm(x, q, pairs, ids, workspace=work), y)
    work.fill_(255)
    out = [torch.full_like(t, float("nan")) for t in (dx, da, db)]
    got = lora.backward(dy, x, q, pairs, ids, out=out, workspace=work)
    for a, b, c in zip(got, out, (dx, da, db)):
        assert a is b and torch.equal(a, c)
    got = lora.backward(dy, None, q, pairs, ids, need_pairs=False)
    assert torch.equal(got[0], dx) and got[1] is None and got[2] is None
    got = lora.backward(dy, x, q, pairs, ids, need_dx=False)
    assert got[0] is None and torch.equal(got[1], da) and torch.equal(got[2], db)


def test_no_rows():
    gen = generator(1)
    q = weight(64, 64, q4.NF4, 64, gen)
    pairs = pairs_of(gen, q4.BF16, 2, 8, 64, 64)
    x = normal(gen, q4.BF16, 0, 64)
    assert lora.gemm(x, q, pairs).shape == (0, 64)
    dx, da, db = lora.backward(x, x, q, pairs)
    assert dx.shape == (0, 64) and not da.any() and not db.any()


def test_captured_and_replayed():
    """With other adapters, ids and activations between replays, eager work beside it."""
    gen = generator(13)
    M, N, K = 130, 96, 128
    q = weight(N, K, q4.NF4, 64, gen)
    pairs = pairs_of(gen, q4.BF16, 3, 16, N, K)
    ids = ids_of(gen, M, 3, "mixed")
    x, dy = normal(gen, q4.BF16, M, K), normal(gen, q4.BF16, M, N)
    few, work, more = x[:5], [torch.empty((lora.workspace_bytes(M, pairs, True),), dtype=torch.uint8, device=DEV)
                              for _ in range(2)], lora.workspace_bytes(5, pairs)
    few_ids = ids[:5]

    def calls():
        return (lora.gemm(x, q, pairs, ids, workspace=work[0]), *lora.backward(dy, x, q, pairs, ids, workspace=work[0]),
                lora.gemm(few, q, pairs, few_ids, workspace=work[1][:more]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = calls()
    for seed in range(4):
        gen = generator(100 + seed)
        pairs.a.copy_(normal(gen, q4.BF16, 3, 16, K, size=K ** -0.5))
        pairs.b.copy_(normal(gen, q4.BF16, 3, N, 16))
        ids.copy_(ids_of(gen, M, 3, "mixed"))
        x.copy_(normal(gen, q4.BF16, M, K))
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        want = (lora.gemm(x, q, pairs, ids), *lora.backward(dy, x, q, pairs, ids), lora.gemm(few, q, pairs, few_ids))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_on_another_stream():
    gen = generator(14)
    M, N, K = 40, 96, 128
    q = weight(N, K, q4.NF4, 64, gen)
    pairs = pairs_of(gen, q4.BF16, 3, 16, N, K)
    ids = ids_of(gen, M, 3, "mixed")
    x, dy = normal(gen, q4.BF16, M, K), normal(gen, q4.BF16, M, N)
    want = (lora.gemm(x, q, pairs, ids), *lora.backward(dy, x, q, pairs, ids))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = (lora.gemm(x, q, pairs, ids), *lora.backward(dy, x, q, pairs, ids))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_outputs_at_any_two_bytes():
    gen = generator(15)
    N, K = 72, 64
    q = weight(N, K, q4.INT4_SYM, 32, gen)
    pairs = pairs_of(gen, q4.BF16, 2, 8, N, K)
    for M in (5, 90, 200, 600):
        x = normal(gen, q4.BF16, M, K)
        flat = torch.full((M * N + 8,), 3.0, dtype=x.dtype, device=DEV)
        check(x, q, pairs, None, out=flat[3:3 + M * N].view(M, N))
        assert bool((flat[:3] == 3).all()) and bool((flat[3 + M * N:] == 3).all())


def test_arguments():
    gen = generator(2)
    q = weight(64, 64, q4.NF4, 64, gen)
    pairs = pairs_of(gen, q4.BF16, 2, 8, 64, 64)
    x = normal(gen, q4.BF16, 6, 64)
    ids = torch.zeros((6,), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        lora.Adapters(pairs.a, pairs.b[:, :, :4].contiguous())
    with pytest.raises(TypeError):
        lora.Adapters(pairs.a.float(), pairs.b.float())
    with pytest.raises(TypeError):
        lora.Adapters(pairs.a, pairs.b.half())
    with pytest.raises(ValueError):
        lora.Adapters(pairs.a, pairs.b, torch.ones((3,), device=DEV))
    with pytest.raises(TypeError):
        lora.gemm(x.half(), q, pairs, ids)
    with pytest.raises(ValueError):
        lora.gemm(x, q, pairs, ids[:5])
    with pytest.raises(TypeError):
        lora.gemm(x, q, pairs, ids.long())
    with pytest.raises(ValueError):
        lora.gemm(x.cpu(), q, pairs)
    with pytest.raises(ValueError):
        lora.gemm(x, weight(128, 64, q4.NF4, 64, gen), pairs)
    with pytest.raises(ValueError):
        lora.backward(x, x[:5], q, pairs)
    moved = lora.Adapters(pairs.a.clone(), pairs.b)
    moved.a.data = pairs.a.clone()
    with pytest.raises(ValueError):
        lora.gemm(x, q, moved)
    with pytest.raises(AttributeError):
        moved.a = pairs.a
    small = torch.empty((lora.workspace_bytes(6, pairs) - 1,), dtype=torch.uint8, device=DEV)
    with pytest.raises(q4.Q4Error) as e:
        lora.gemm(x, q, pairs, workspace=small)
    assert e.value.status == q4.EINVAL
    assert ctypes.sizeof(lora._LoraArgs) == 40


@pytest.mark.parametrize("part", ["a", "b", "scale"])
def test_tensors_replaced_under_the_adapters(part):
    """Another storage, shape or type behind a tensor's name is refused, and the first one's memory is not given away."""
    gen = generator(17)
    q = weight(64, 64, q4.NF4, 64, gen)
    x = normal(gen, q4.BF16, 6, 64)

    def made():
        pairs = pairs_of(gen, q4.BF16, 2, 8, 64, 64)
        lora.gemm(x, q, pairs)
        return pairs, getattr(pairs, part)

    def refused(pairs):
        with pytest.raises(ValueError):
            lora.gemm(x, q, pairs)
        with pytest.raises(ValueError):
            lora.backward(x, x, q, pairs)

    pairs, t = made()
    kept = t.clone()
    t.mul_(0.5)  # (values may change)
    lora.gemm(x, q, pairs)
    old = t.data_ptr()
    t.data = kept
    refused(pairs)
    others = [torch.empty_like(kept) for _ in range(64)]
    assert old not in [o.data_ptr() for o in others]
    pairs, t = made()
    t.set_(torch.empty_like(t))
    refused(pairs)
    pairs, t = made()
    t.data = t.data.reshape(-1)[:t.numel() // 2]
    refused(pairs)
    pairs, t = made()
    t.data = t.data.view(torch.int32 if part == "scale" else torch.float16)
    refused(pairs)


def test_each_gradient_of_no_rows_alone():
    gen = generator(1)
    q = weight(64, 128, q4.NF4, 64, gen)
    pairs = pairs_of(gen, q4.BF16, 2, 8, 64, 128)
    x, dy = normal(gen, q4.BF16, 0, 128), normal(gen, q4.BF16, 0, 64)
    dx, da, db = lora.backward(dy, None, q, pairs, need_pairs=False)
    assert dx.shape == (0, 128) and da is None and db is None
    out = (None, torch.ones_like(pairs.a), torch.ones_like(pairs.b))
    dx, da, db = lora.backward(dy, x, q, pairs, need_dx=False, out=out)
    assert dx is None and not da.any() and not db.any()


@pytest.mark.parametrize("rank", [8, 72, 256])
@pytest.mark.parametrize("name", list(LORA))
def test_each_kernel(name, rank):
    """Mixed adapters and none, an adapter that is not finite, a row of NaN, outputs at any element."""
    _, M, N, K, g = LORA[name]
    gen = generator(M + N + rank)
    for act in (q4.F16, q4.BF16):
        q = weight(N, K, FORMATS[(len(name) + rank // 8 + act) % 5], g, gen)
        pairs = pairs_of(gen, act, 5, rank, N, K)
        ids = ids_of(gen, M, 5, "mixed")
        bad = M // 2
        ids[0], ids[bad] = 1, 4
        x = normal(gen, act, M, K)
        y = check(x, q, pairs, ids, name)
        flat = torch.full((M * N + 16,), 3.0, dtype=x.dtype, device=DEV)
        got = lora.gemm(x, q, pairs, ids, out=flat[1:1 + M * N].view(M, N))
        assert torch.equal(got, y) and bool((flat[:1] == 3).all()) and bool((flat[1 + M * N:] == 3).all())
        x[bad] = float("nan")
        pairs.a[3], pairs.b[3] = float("nan"), float("inf")
        keep = (ids != 3) & (torch.arange(M, device=DEV) != bad)
        got = lora.gemm(x, q, pairs, ids)
        assert torch.equal(got[keep], y[keep]) and bool(torch.isnan(got[bad]).all())
        assert not bool((ids == 3).any()) or not bool(torch.isfinite(got[ids == 3]).any())


@pytest.mark.parametrize("rank", [16, 136])
@pytest.mark.parametrize("name", list(LORA_DX))
@pytest.mark.parametrize("fmt", FORMATS)
def test_each_gradient_kernel(fmt, name, rank):
    _, _, M, N, K, g = LORA_DX[name]
    gen = generator(M + N + rank)
    act = (fmt + rank // 8) % 2
    q = weight(N, K, fmt, g, gen)
    pairs = pairs_of(gen, act, 3, rank, N, K)
    ids = ids_of(gen, M, 3, "mixed")
    check_backward(normal(gen, act, M, N), normal(gen, act, M, K), q, pairs, ids, name)


def test_kernels_captured_and_replayed():
    """The wide tiles, with other ids and adapters between replays."""
    for name in ("tile128", "tile256", "skinny-blocks3"):
        _, M, N, K, g = LORA[name]
        gen = generator(N)
        q = weight(N, K, q4.INT4_ASYM, g, gen)
        pairs = pairs_of(gen, q4.BF16, 3, 24, N, K)
        ids, x = ids_of(gen, M, 3, "mixed"), normal(gen, q4.BF16, M, K)
        work = torch.empty((lora.workspace_bytes(M, pairs),), dtype=torch.uint8, device=DEV)
        out = x.new_empty((M, N))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lora.gemm(x, q, pairs, ids, out=out, workspace=work)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lora.gemm(x, q, pairs, ids, out=out, workspace=work)
        for seed in range(3):
            gen = generator(200 + seed)
            pairs.b.copy_(normal(gen, q4.BF16, 3, N, 24))
            ids.copy_(ids_of(gen, M, 3, "mixed"))
            x.copy_(normal(gen, q4.BF16, M, K))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, check(x, q, pairs, ids, name))


def whole(gen, act, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV).to(ACTS[act])


def nearly_twice(t, dim):
    """Every second slice of t along dim made the one before it, but for two of its values that are one larger."""
    t = t.movedim(dim, 0).clone()
    for odd in range(1, t.shape[0], 2):
        t[odd] = t[odd - 1]
        flat = t[odd].reshape(-1, t.shape[-1])
        flat[:, (5 * odd) % t.shape[-1]] += 1
        flat[:, (7 * odd + 3) % t.shape[-1]] += 1
    return t.movedim(0, dim).contiguous()


def differences(act, rows, columns):
    """[rows, columns] (rows even) with 1 in an even row and -1 in the next, a pair of rows for each column."""
    t = torch.zeros((rows, columns), dtype=ACTS[act], device=DEV)
    c = torch.arange(columns, device=DEV)
    even = 2 * (c % (rows // 2))
    t[even, c], t[even + 1, c] = 1, -1
    return t


def largest(n):
    """Of the whole numbers in a sum of n: its terms' mean makes sums of 2^18 to 2^20."""
    return max(4, min(62, 6000 // n))


@pytest.mark.parametrize("rank", [8, 24, 40, 136])
@pytest.mark.parametrize("name", ["skinny", "skinny-two", "skinny-four", "tile64", "tile64-parts", "tile128", "tile256"])
def test_every_bit_of_the_low_product(name, rank):
    """Whole numbers, exact in binary32: h of 2^18 and more, whose small differences y has to hold exactly."""
    _, M, N, K, g = LORA[name]
    gen = generator(M + rank)
    for act in (q4.F16, q4.BF16):
        q = q4.quantize(torch.zeros((N, K), dtype=torch.float16, device=DEV), q4.INT4_SYM, g)
        x = whole(gen, act, 1, largest(K), M, K)
        a = nearly_twice(whole(gen, act, 64, 126, 1, rank, K), 1)
        b = differences(act, rank, N).t().contiguous()[None]
        h = x.double() @ a[0].double().T
        assert float(h.abs().max()) > 2 ** 18 and float(h.abs().max()) < 2 ** 24
        y = lora.gemm(x, q, lora.Adapters(a, b))
        assert torch.equal(y.double(), h @ b[0].double().T) and bool((y != 0).any())


@pytest.mark.parametrize("rank", [8, 24, 40, 136])
@pytest.mark.parametrize("name", list(LORA_DX))
def test_every_bit_of_the_low_products_gradients(name, rank):
    """The same for u in dx (whose A takes differences of values r), and for h and u in db and da (whose dy and x take
    differences of rows)."""
    _, _, M, N, K, g = LORA_DX[name]
    M -= M % 2
    gen = generator(M + rank)
    for act in (q4.F16, q4.BF16):
        q = q4.quantize(torch.zeros((N, K), dtype=torch.float16, device=DEV), q4.INT4_SYM, g)
        b = nearly_twice(whole(gen, act, 64, 126, 1, N, rank), 2)
        pairs = lora.Adapters(differences(act, rank, K)[None].contiguous(), b)
        dy = whole(gen, act, 1, largest(N), M, N)
        u = dy.double() @ b[0].double()
        assert float(u.abs().max()) > 2 ** 17 and float(u.abs().max()) < 2 ** 24
        dx, _, _ = lora.backward(dy, None, q, pairs, need_pairs=False)
        assert torch.equal(dx.double(), u @ pairs.a[0].double()) and bool((dx != 0).any())

        dy, x = nearly_twice(dy, 0), differences(act, M, K)
        u = dy.double() @ b[0].double()
        _, da, _ = lora.backward(dy, x, q, pairs, need_dx=False)
        want = u.T @ x.double()
        assert float(want.abs().max()) <= 256 and torch.equal(da[0].double(), want) and bool((da != 0).any())

        x, dy = nearly_twice(whole(gen, act, 1, largest(K), M, K), 0), differences(act, M, N)
        a = whole(gen, act, 64, 126, 1, rank, K)
        h = x.double() @ a[0].double().T
        _, _, db = lora.backward(dy, x, q, lora.Adapters(a, b), need_dx=False)
        want = dy.double().T @ h
        assert float(want.abs().max()) <= 256 and torch.equal(db[0].double(), want) and bool((db != 0).any())


def assert_same_kind(got, want, tag):
    """NaN where the formula is, infinities of its sign, numbers elsewhere."""
    got = got.double()
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(got), kind(want)), f"{tag} {kind.__name__}"


@pytest.mark.parametrize("rank", [8, 72])
@pytest.mark.parametrize("name", ["skinny", "skinny-two", "skinny-four", "tile64", "tile64-parts", "tile128", "tile256"])
def test_infinities_of_adapters(name, rank):
    """An infinite value of A or B: infinities and NaN as the formula has them, beside values that 8 bits hold and others."""
    _, M, N, K, g = LORA[name]
    gen = generator(M + rank)
    for act in (q4.F16, q4.BF16):
        q = weight(N, K, q4.NF4, g, gen)
        x = normal(gen, act, M, K)
        x[::2] = whole(gen, act, -3, 3, (M + 1) // 2, K)
        a, b = whole(gen, act, -2, 2, 3, rank, K), normal(gen, act, 3, N, rank)
        a[2], b[1] = normal(gen, act, rank, K), whole(gen, act, -2, 2, N, rank)
        a[0, 5, 7], a[1, rank - 1, 3] = float("inf"), -float("inf")
        b[1, N // 2, 2], b[2, N - 1, 6], b[2, 0, 1] = float("inf"), -float("inf"), float("inf")
        ids = ids_of(gen, M, 3, "mixed")
        ids[:4] = torch.tensor([0, 1, 2, 0], device=DEV)
        y = lora.gemm(x, q, lora.Adapters(a, b), ids)
        want = x.double() @ values(q, act).T
        for i in range(3):
            at = (ids == i).nonzero()[:, 0]
            want[at] += (x[at].double() @ a[i].double().T) @ b[i].double().T
        assert bool(torch.isinf(want).any())
        assert_same_kind(y, want, name)


@pytest.mark.parametrize("rank", [8, 24, 72])
@pytest.mark.parametrize("name", list(LORA_DX))
def test_infinities_of_adapters_in_gradients(name, rank):
    _, _, M, N, K, g = LORA_DX[name]
    gen = generator(M + rank)
    inf = float("inf")
    for act in (q4.F16, q4.BF16):
        q = weight(N, K, q4.NF4, g, gen)
        x, dy = normal(gen, act, M, K), normal(gen, act, M, N)
        x[::2], dy[::3] = whole(gen, act, -3, 3, (M + 1) // 2, K), whole(gen, act, -3, 3, (M + 2) // 3, N)
        a, b = whole(gen, act, -2, 2, 3, rank, K), normal(gen, act, 3, N, rank)
        a[2], b[1] = normal(gen, act, rank, K), whole(gen, act, -2, 2, N, rank)
        a[0, 5, 7], b[1, N // 2, 2], b[2, 3, 6] = inf, -inf, inf
        ids = torch.full((M,), -1, dtype=torch.int32, device=DEV)
        ids[M // 2], ids[M // 3], ids[M - 1], ids[1] = 0, 1, 2, 2
        dx, da, db = lora.backward(dy, x, q, lora.Adapters(a, b), ids)
        want = dy.double() @ values(q, act)
        for i in range(3):
            at = (ids == i).nonzero()[:, 0]
            u, h = dy[at].double() @ b[i].double(), x[at].double() @ a[i].double().T
            want[at] += u @ a[i].double()
            assert_same_kind(da[i], u.T @ x[at].double(), f"{name} da {i}")
            assert_same_kind(db[i], dy[at].double().T @ h, f"{name} db {i}")
        assert bool(torch.isinf(want).any()) and not bool(torch.isfinite(db[0]).all() or torch.isfinite(da[2]).all())
        assert_same_kind(dx, want, f"{name} dx")


@pytest.mark.parametrize("M,N,K,adapters,rank", [
    (5, 520, 4096, 3, 16), (95, 1000, 2048, 8, 72),                 # h in parts
    (200, 2056, 5888, 3, 72), (130, 1032, 1024, 2, 8),              # and K, N in parts
    (2048, 264, 2048, 8, 32), (4100, 136, 1280, 1, 64), (5000, 256, 512, 1, 64),  # and the rows
    (300, 72, 96, 5, 256)])
def test_a_workspace_of_exactly_the_bytes(M, N, K, adapters, rank):
    """Nothing behind it is written or matters, and nothing in it before."""
    gen = generator(M + N)
    for act in (q4.F16, q4.BF16):
        q = weight(N, K, q4.NF4, 32, gen)
        pairs = pairs_of(gen, act, adapters, rank, N, K)
        ids = ids_of(gen, M, adapters, "mixed")
        x, dy = normal(gen, act, M, K), normal(gen, act, M, N)
        for bwd in (False, True):
            n = lora.workspace_bytes(M, pairs, bwd)
            room = torch.full((n + 65536,), 255, dtype=torch.uint8, device=DEV)
            call = check_backward if bwd else check
            given = (dy, x) if bwd else (x,)
            first = call(*given, q, pairs, ids, workspace=room[:n])
            assert bool((room[n:] == 255).all())
            room[n:] = 0
            again = call(*given, q, pairs, ids, workspace=room[:n])
            for a, b in zip(first, again) if bwd else ((first, again),):
                assert torch.equal(a, b)
