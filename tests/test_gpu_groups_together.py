"""Grouped products together, as a fine-tuning step of a mixture uses them: a
projection with adapters, routed to experts (gathered rows, gate and up, down),
combined, and the gradients back through the experts to the adapters, which an
update then changes.  Every stage is held to the formula in binary64 on the
16-bit tensors that it was given."""

import pytest
import torch

from bit_group_wise_amd import experts, lora, q4
from _groups import ACTS, DEV, generator, half_step, normal, values, weight

pytestmark = pytest.mark.gpu


def near(got, want, sums, act, tag):
    """`sums` bounds the error of the binary32 sums and of 16-bit second operands; the output is rounded once."""
    if got.numel() == 0:
        return
    worst = ((got.double() - want).abs() - (sums + half_step(act) * (want.abs() + sums) + 2.0 ** -25)).max()
    assert float(worst) <= 0, f"{tag}: {float(worst)}"


@pytest.mark.parametrize("fmt,act,tokens", [(q4.NF4, q4.BF16, 7), (q4.INT4_ASYM, q4.BF16, 150),
                                            (q4.NF4_DQ, q4.F16, 700)])
def test_a_step_of_a_mixture_with_adapters(fmt, act, tokens):
    gen = generator(tokens)
    D, I, E, top, R, A = 192, 256, 6, 2, 16, 2
    proj = weight(D, D, fmt, 64, gen)
    up, down = weight(E * 2 * I, D, fmt, 64, gen), weight(E * D, I, fmt, 64, gen)
    pairs = lora.Adapters(normal(gen, act, A, R, D, size=D ** -0.5), normal(gen, act, A, D, R, size=0.1),
                          torch.tensor([2.0, 0.5], device=DEV))
    ids = torch.randint(-1, A, (tokens,), generator=gen, device=DEV).int()
    x = normal(gen, act, tokens, D)
    target = normal(gen, act, tokens, D)
    wp, wu, wd = values(proj, act), values(up, act).view(E, 2 * I, D), values(down, act).view(E, D, I)
    short = lambda n: n * 2.0 ** -23  # noqa: E731

    # routing by a table of chance; each token's copies sorted by expert
    score = torch.rand((tokens, E), generator=gen, device=DEV)
    gate, who = score.topk(top, dim=1)
    gate = (gate / gate.sum(1, keepdim=True)).to(ACTS[act])
    order = who.reshape(-1).argsort(stable=True)
    index = (order // top).int()
    offsets = torch.nn.functional.pad(torch.bincount(who.reshape(-1), minlength=E).cumsum(0), (1, 0)).int()
    expert = who.reshape(-1)[order]

    losses = []
    for step in range(2):
        h = lora.gemm(x, proj, pairs, ids)
        gu = experts.gemm(h, up, offsets, index=index)
        g, u = gu[:, :I].float(), gu[:, I:].float()
        s = torch.sigmoid(g)
        act_rows = (g * s * u).to(h.dtype)
        rows = experts.gemm(act_rows, down, offsets)
        weighed = rows.float() * gate.reshape(-1)[order].float()[:, None]
        y = torch.zeros((tokens, D), device=DEV).index_add_(0, index.long(), weighed)
        dy = (y - target.float()).to(h.dtype)
        losses.append(float((y - target.float()).square().mean()))
        drows = (dy.float()[index.long()] * gate.reshape(-1)[order].float()[:, None]).to(h.dtype)
        dact = experts.gemm_dx(drows, down, offsets)
        dg = dact.float() * u * (s + g * s * (1 - s))
        dgu = torch.cat((dg, dact.float() * g * s), 1).to(h.dtype)
        dcopies = experts.gemm_dx(dgu, up, offsets)
        dh = torch.zeros((tokens, D), device=DEV).index_add_(0, index.long(), dcopies.float()).to(h.dtype)
        dx, da, db = lora.backward(dh, x, proj, pairs, ids)

        # every stage against its formula
        def through(name, got, rows_in, w, transposed):
            a = rows_in.double()
            for e in range(E):
                at = (expert == e).nonzero()[:, 0]
                we = w[e] if transposed else w[e].T
                near(got[at], a[at] @ we, short(a.shape[1] + 1) * (a[at].abs() @ we.abs()), act, f"{name} {e}")

        through("gate and up", gu, h[index.long()], wu, False)
        through("down", rows, act_rows, wd, False)
        through("down's gradient", dact, drows, wd, True)
        through("gate and up's gradient", dcopies, dgu, wu, True)
        want, wantd = x.double() @ wp.T, dh.double() @ wp
        sums, sumsd = short(D + 1) * (x.double().abs() @ wp.abs().T), short(D + 1) * (dh.double().abs() @ wp.abs())
        for i in range(A):
            at = (ids == i).nonzero()[:, 0]
            a, b, sc = pairs.a[i].double(), pairs.b[i].double(), float(pairs.scale[i])
            xr, dr = x[at].double(), dh[at].double()
            hid, u64 = sc * xr @ a.T, sc * dr @ b
            habs, uabs = sc * xr.abs() @ a.abs().T, sc * dr.abs() @ b.abs()
            want[at] += hid @ b.T
            wantd[at] += u64 @ a
            sums[at] += (habs @ b.abs().T) * (short(D + 4 * R) + 2.0 ** -17)
            sumsd[at] += (uabs @ a.abs()) * (short(D + 4 * R) + 2.0 ** -17)
            more = short(D + 3 * len(at) + 16) + 2.0 ** -17
            near(da[i], u64.T @ xr, (uabs.T @ xr.abs()) * more, act, f"da {i}")
            near(db[i], dr.T @ hid, (dr.abs().T @ habs) * more, act, f"db {i}")
        near(h, want, sums, act, "projection")
        near(dx, wantd, sumsd, act, "projection's gradient")

        # the adapters' step (the next round's products see it)
        before = h.clone()
        pairs.a.sub_(1e-2 * da / da.float().norm().clamp(min=1e-6).to(da.dtype))
        pairs.b.sub_(1e-2 * db / db.float().norm().clamp(min=1e-6).to(db.dtype))
        if step == 0 and bool((ids >= 0).any()):
            assert not torch.equal(lora.gemm(x, proj, pairs, ids), before)
    assert all(torch.isfinite(torch.tensor(losses)))
