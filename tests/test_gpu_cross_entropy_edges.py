"""Softmax cross entropy where sizes, addresses and logits are at their ends (tolerances: those of test_gpu_cross_entropy)."""
import math

import pytest
import torch

from test_gpu_cross_entropy import BF, DTS, F, U24, UNIT, _case, _check, _close, _gen
from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("R", [1, 3, 64, 65, 300])
@pytest.mark.parametrize("D", [64, 200, 264])
@pytest.mark.parametrize("z", [-1000.0, 1000.0])
def test_one_item_is_always_right(z, D, R, dt):
    """A vocabulary of one item: the loss and its gradients are 0, however far its logit is from 0."""
    H, E = torch.ones(R, D, device="cuda", dtype=dt), torch.full((1, D), z / D, device="cuda").to(dt)
    loss, rows, saved = ops.cross_entropy_forward(H, E, torch.zeros(R, dtype=torch.int32, device="cuda"))
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    alone = ops.cross_entropy_forward(H, E, torch.zeros(R, dtype=torch.int32, device="cuda"), want_grad=False)[0]
    for x in (loss, rows, dH, dE, alone):
        assert torch.equal(x, torch.zeros_like(x))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("D", [64, 128, 256, 264])
def test_all_logits_far_from_zero(D, dt):
    """Logits about -1000 or 1000: only their differences count."""
    for z in (-1000.0, 1000.0):
        H, E, t, w = _case(70, 900, D, dt, seed=50, lean=0.0)
        H[:, 0], E[:, 0] = 1.0, z
        _check(H, E, t, w)


@pytest.mark.parametrize("D", [32, 200, 256])
def test_logits_that_rise(D):
    """References that do not hold: logits that rise by 60 and by 600 along the items."""
    t = _case(130, 2000, D, BF, seed=4)[2]
    ramp = torch.linspace(-1, 1, 2000, device="cuda")[:, None]
    for k in (30.0, 300.0):
        for sign in (1.0, -1.0):
            E = (sign * k * ramp * torch.ones(1, D, device="cuda") / D).to(BF)
            H = (torch.ones(130, D, device="cuda") + 0.1 * torch.randn(130, D, generator=_gen(5), device="cuda")).to(BF)
            _check(H, E, t)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("R", [15, 16, 17, 63, 64, 65, 1023, 1024, 1025, 8192, 8193, 8200])
def test_numbers_of_rows(R, dt):
    for D in (64, 264):
        H, E, t, w = _case(R, 130, D, dt, seed=R, left_out=0.5, id_dt=torch.int64)
        _check(H, E, t, w)


@pytest.mark.parametrize("dt,D", [(BF, 64), (BF, 264), (F, 40)])
def test_a_million_rows(dt, D):
    """The most rows that a call takes; most of them are left out."""
    R, V = 1 << 20, 70
    H, E, t, w = _case(R, V, D, dt, seed=60, left_out=0.9)
    _check(H, E, t, w)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("D", [64, 264])
def test_addresses_and_strides(D, dt):
    """Rows that begin in the middle of 16 bytes, with gaps, transposed, or one row many times."""
    H, E, t, w = _case(90, 300, D, dt, seed=61)
    def moved(x):
        y = torch.empty(x.numel() + 1, dtype=dt, device="cuda")[1:].view(x.shape)
        y.copy_(x)
        return y
    want = ops.cross_entropy_forward(H, E, t, w)
    g = torch.ones(1, device="cuda")
    grads = ops.cross_entropy_backward(g, H, E, want[2])
    wide = torch.zeros(300, 2 * D, dtype=dt, device="cuda")
    wide[:, ::2] = E
    every = torch.zeros(180, dtype=t.dtype, device="cuda")
    every[::2] = t
    for h, e, tt in ((moved(H), moved(E), t), (H.T.contiguous().T, wide[:, ::2], every[::2])):
        got = ops.cross_entropy_forward(h, e, tt, w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, ops.cross_entropy_backward(g, h, e, got[2])))
    _check(H[:1].expand(90, D), E, t, w)
    one = H[:1].clone().requires_grad_()
    ops.cut_cross_entropy(one.expand(90, D), E, t, w).backward()
    same = H[:1].expand(90, D).contiguous()
    per = ops.cross_entropy_backward(g, same, E, ops.cross_entropy_forward(same, E, t, w)[2])[0]
    assert torch.allclose(one.grad.double(), per.double().sum(0, keepdim=True), rtol=2 * UNIT[dt], atol=2 * UNIT[dt] * per.abs().double().sum(0).max().item())


@pytest.mark.parametrize("V,D", [(9_000_001, 256), (4_500_001, 512)])
def test_offsets_past_32_bits(V, D):
    """More than 2^32 bytes of items, most of them zeros (logit 0, so that sums are known): the loss, and dE at the array's
    ends and in its middle. Sums of 9 million equal numbers are off by u (V / 64 + 128) at worst."""
    R = 24
    E = torch.zeros(V, D, dtype=BF, device="cuda")
    some = torch.cat([torch.arange(40), torch.arange(V // 2, V // 2 + 40), torch.arange(V - 40, V)]).cuda()
    E[some] = (torch.randn(some.numel(), D, generator=_gen(70), device="cuda") * 3 / math.sqrt(D)).to(BF)
    t = some[torch.randint(0, some.numel(), (R,), generator=_gen(71), device="cuda")].to(torch.int32)
    H = (torch.randn(R, D, generator=_gen(72), device="cuda")).to(BF)
    loss, rows, saved = ops.cross_entropy_forward(H, E, t)
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    h, e = H.double(), E[some].double()
    z = h @ e.T.contiguous()
    lse = torch.log(torch.exp(z).sum(1) + (V - some.numel()))
    at = (some[None] == t[:, None]).double()
    zt = (z * at).sum(1)
    chain = U24 * (V / 64 + 128) + 1e-5
    _close("row_loss", rows, lse - zt, torch.full_like(lse, chain))
    _close("loss", loss, (lse - zt).mean(), torch.full((), chain, device="cuda", dtype=torch.float64))
    p = (torch.exp(z - lse[:, None]) - at) / R
    off = (p.abs() * (UNIT[BF] + chain)).T.contiguous() @ h.abs() + 2.0 ** -126 * h.abs().sum(0)
    want = p.T.contiguous() @ h
    _close("dE", dE[some], want, off + UNIT[BF] * (want.abs() + off))
    zero = torch.exp(-lse) / R
    want = (zero @ h).expand(3, D)
    off = ((zero * (UNIT[BF] + chain)) @ h.abs()).expand(3, D) + 2.0 ** -126 * h.abs().sum(0)
    _close("dE of zeros", dE[torch.tensor([41, V // 2 - 1, V - 41], device="cuda")], want, off + UNIT[BF] * (want.abs() + off))
    want = p @ e
    off = (p.abs() * (UNIT[BF] + chain)) @ e.abs() + 2.0 ** -126 * e.abs().sum(0)
    _close("dH", dH, want, off + UNIT[BF] * (want.abs() + off))


@pytest.mark.parametrize("left_out", [0.0, 0.2])
@pytest.mark.parametrize("R,V,D,dt", [(600, 500, 8192, F), (600, 500, 8192, BF), (2100, 7500, 2000, BF), (700, 70_000, 264, BF),
                                      (64, 30_000, 272, F), (64, 30_000, 520, BF)])
def test_long_axes_in_parts(R, V, D, dt, left_out):
    """Tiles of dH that do not fill whole turns of the chip, or few of them with many parts; how many depends on the rows
    that are counted."""
    H, E, t, w = _case(R, V, D, dt, seed=R + D, left_out=left_out)
    _check(H, E, t, w)
