"""Adapters beside a projection, their gradients, 8-bit checkpoints and the input gradient on the GPU,
against the float64 oracle with its derived bounds."""

import numpy as np
import pytest
import torch

import oracle
from oracle import adapter_oracle as ao

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def cr():
    import w4a8_rotated_quantized_b200 as m

    return m


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(BF)


def strided(t, pad):
    """The same matrix with rows `pad` elements further apart, the gap filled with NaN."""
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def rows_of(mix, M, L, g):
    if mix == "all":
        return None
    if mix == "none":
        return torch.full((M,), -1, dtype=torch.int32, device="cuda")
    if mix == "rows":  # any order, some outside the pool on either side
        return torch.randint(-2, L + 2, (M,), device="cuda", generator=g, dtype=torch.int32)
    if mix == "last":  # one row only, the last
        a = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        a[-1] = L - 1
        return a
    # runs: one after the other, padding behind the last
    cuts = torch.sort(torch.randint(0, M + 1, (L,), device="cuda", generator=g)).values
    a = torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True).to(torch.int32)
    return torch.where(a >= L, torch.full_like(a, -1), a)


def make(M, K, N, r, L, mix, seed=0):
    g = gen(seed)
    return dict(X=randn(g, M, K), down=randn(g, L, r, K, std=K ** -0.5), up=randn(g, L, r, N, std=0.05),
                scale=0.25 + torch.rand(L, device="cuda", generator=g), adapter=rows_of(mix, M, L, g),
                base=randn(g, M, N), dY=randn(g, M, N, std=1e-2), dbase=randn(g, M, K, std=1e-2))


def within(got, want, bound, what):
    got = f64(got).reshape(want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - want) - bound
    assert off.max(initial=-1) <= 0, f"{what}: over its bound by {off.max():.3g} at {np.unravel_index(off.argmax(), off.shape)}"


def ids(a):
    return None if a is None else a.cpu().numpy()


SHAPES = [  # M, K, N, rank, adapters, rows
    (1, 2560, 9728, 16, 1, "all"),
    (1, 8, 8, 4, 1, "all"),
    (3, 264, 72, 12, 2, "rows"),
    (16, 2560, 1000, 8, 5, "rows"),
    (17, 512, 256, 100, 3, "rows"),
    (64, 1032, 520, 16, 48, "rows"),
    (65, 768, 2056, 128, 2, "runs"),
    (128, 256, 264, 20, 7, "rows"),
    (129, 512, 256, 64, 2, "last"),
    (130, 9728, 2560, 32, 3, "runs"),
    (300, 640, 384, 4, 300, "rows"),
    (513, 512, 512, 36, 9, "runs"),
    (777, 512, 256, 8, 5, "runs"),
    (1100, 3072, 1544, 64, 1, "all"),
    (2049, 1280, 776, 128, 4, "runs"),
    (1500, 264, 1032, 12, 40, "rows"),
    (1300, 256, 520, 128, 9, "rows"),
    (9, 65536, 8, 4, 2, "rows"),
    (70, 32768, 16, 8, 70, "rows"),
    (3, 256, 65536, 8, 2, "rows"),
    (200, 256, 256, 16, 3, "none"),
    (40, 256, 256, 32, 20, "none"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape):
    d = make(*shape, seed=1)
    want, v, ey, ev = ao.lora_forward(f64(d["X"]), f64(d["down"]), f64(d["up"]), f64(d["scale"]), ids(d["adapter"]),
                                      f64(d["base"]))
    Y, V = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], base=d["base"],
                                save_v=True)
    within(Y, want, ey, "Y")
    within(V, v, ev, "V")
    Y2 = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], base=d["base"])
    assert torch.equal(Y.view(torch.int16), Y2.view(torch.int16))


@pytest.mark.parametrize("has_base", [True, False])
@pytest.mark.parametrize("r,L,mix", [(24, 5, "runs"), (128, 9, "runs"), (64, 6, "rows"), (16, 2, "last"), (100, 1, "all"), (4, 3, "none")])
def test_column_tiles_dealt_out_over_token_tiles(r, L, mix, has_base):
    """75 token tiles of 20 column tiles: most CTAs go on from one token tile to the next."""
    d = make(9500, 136, 2504, r, L, mix, seed=9)
    base = d["base"] if has_base else None
    args = (d["down"], d["up"], d["scale"])
    want, _, ey, _ = ao.lora_forward(f64(d["X"]), *(f64(t) for t in args), ids(d["adapter"]), f64(base) if has_base else None)
    got = cr().cr_lora_forward(d["X"], *args, adapter=d["adapter"], base=base)
    within(got, want, ey, "Y")
    parts = [cr().cr_lora_forward(d["X"][i:j], *args, adapter=None if d["adapter"] is None else d["adapter"][i:j],
                                  base=base[i:j] if has_base else None) for i, j in ((0, 2048), (2048, 9500))]
    assert torch.equal(got, torch.cat(parts))


@pytest.mark.parametrize("shape", [(5, 264, 136, 8, 2, "rows"), (150, 520, 264, 24, 3, "runs"), (1, 256, 64, 4, 1, "all")],
                         ids=str)
def test_forward_strides_no_base_and_in_place(shape):
    d = make(*shape, seed=2)
    X = strided(d["X"], 24)
    args = (d["down"], d["up"], d["scale"])
    plain = cr().cr_lora_forward(d["X"], *args, adapter=d["adapter"], base=d["base"])
    big = strided(d["base"].clone(), 40)
    whole = big._base if big._base is not None else big
    gap = whole[:, d["base"].shape[1]:].clone()
    got = cr().cr_lora_forward(X, *args, adapter=d["adapter"], base=big, out=big)
    assert got is big and torch.equal(got, plain)
    assert torch.equal(whole[:, d["base"].shape[1]:].view(torch.int16), gap.view(torch.int16))  # between the rows: untouched
    want, _, ey, _ = ao.lora_forward(f64(d["X"]), *(f64(t) for t in args), ids(d["adapter"]))
    within(cr().cr_lora_forward(X, *args, adapter=d["adapter"]), want, ey, "Y without base")


@pytest.mark.parametrize("M", [24, 200, 600])
def test_values_stay_in_their_rows(M):
    """NaN and infinities in one row, in one adapter or in rows without adapter change nothing else."""
    d = make(M, 512, 264, 16, 4, "rows", seed=3)
    a = d["adapter"]
    a[:5] = torch.tensor([0, 1, 2, 3, -1], device="cuda")
    args = dict(adapter=a, base=d["base"])
    Y0, V0 = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], save_v=True, **args)
    X, down, up = d["X"].clone(), d["down"].clone(), d["up"].clone()
    X[1, 7], X[4, :] = float("inf"), float("nan")
    down[2, 3, 5], up[2, 1, :] = float("nan"), float("inf")
    Y, V = cr().cr_lora_forward(X, down, up, d["scale"], save_v=True, **args)
    ok = (a != 2)
    ok[1] = False
    assert torch.equal(Y[ok].view(torch.int16), Y0[ok].view(torch.int16))
    assert torch.equal(V[ok].view(torch.int16), V0[ok].view(torch.int16))
    assert not torch.isfinite(Y[1]).any() and not torch.isfinite(Y[a == 2]).any()
    # gradients: rows without adapter, and adapter 2's rows, hold NaN; the others' gradients are as before
    none = ~((a >= 0) & (a < 4))
    dY = d["dY"]
    g0 = cr().cr_lora_backward(dY, d["X"], V0, d["down"], d["up"], d["scale"], adapter=a, base=d["dbase"])
    c0 = cr().cr_ckpt_save(d["X"])
    h0 = cr().cr_lora_backward(dY, c0, V0, d["down"], d["up"], d["scale"], adapter=a, base=d["dbase"])
    bad = none | (a == 2)
    Xb, dYb, Vb = d["X"].clone(), dY.clone(), V0.clone()
    Xb[bad], dYb[bad], Vb[bad] = float("nan"), float("inf"), float("nan")
    cb = cr().cr_ckpt_save(Xb)
    assert torch.isnan(cb[1][bad]).all() and torch.isfinite(cb[1][~bad]).all()
    for kept, ref in ((Xb, g0), (cb, h0)):
        dX, dd, du = cr().cr_lora_backward(dYb, kept, Vb, d["down"], d["up"], d["scale"], adapter=a, base=d["dbase"])
        assert torch.equal(dX[~bad].view(torch.int16), ref[0][~bad].view(torch.int16))
        assert torch.equal(dX[none].view(torch.int16), d["dbase"][none].view(torch.int16))
        for x, y in ((dd, ref[1]), (du, ref[2])):
            assert torch.equal(x[[0, 1, 3]].view(torch.int16), y[[0, 1, 3]].view(torch.int16))
        assert not torch.isfinite(dd[2]).all() and not torch.isfinite(du[2]).all()


@pytest.mark.parametrize("kept", ["bf16", "int8"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] != 1] + [(1, 512, 256, 16, 1, "all"), (5000, 256, 264, 8, 3, "runs")],
                         ids=str)
def test_backward(shape, kept):
    M, K, N, r, L, mix = shape
    if kept == "int8":
        K = max(256, K // 256 * 256)
    d = make(M, K, N, r, L, mix, seed=4)
    _, V = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], save_v=True)
    if kept == "int8":
        keep = cr().cr_ckpt_save(d["X"])
        x, mags = ao.ckpt_values(keep[0].cpu().numpy(), keep[1].cpu().numpy())
    else:
        keep, x, mags = d["X"], f64(d["X"]), None
    want, bound = ao.lora_backward(f64(d["dY"]), x, f64(V), f64(d["down"]), f64(d["up"]), f64(d["scale"]),
                                   ids(d["adapter"]), f64(d["dbase"]), mags)
    args = (d["dY"], keep, V, d["down"], d["up"], d["scale"])
    got = cr().cr_lora_backward(*args, adapter=d["adapter"], base=d["dbase"])
    for g, w, b, name in zip(got, want, bound, ("dX", "d_down", "d_up")):
        within(g, w, b, name)
    again = cr().cr_lora_backward(*args, adapter=d["adapter"], base=d["dbase"])
    for x1, x2 in zip(got, again):
        assert torch.equal(x1.view(torch.int16), x2.view(torch.int16))


def test_backward_parts_strides_and_in_place():
    d = make(333, 512, 264, 24, 3, "runs", seed=5)
    _, V = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], save_v=True)
    tail = (d["down"], d["up"], d["scale"])
    want = cr().cr_lora_backward(d["dY"], d["X"], V, *tail, adapter=d["adapter"], base=d["dbase"])
    base = strided(d["dbase"].clone(), 8)
    got = cr().cr_lora_backward(strided(d["dY"], 16), strided(d["X"], 24), V, *tail, adapter=d["adapter"], base=base,
                                out=base)
    assert got[0] is base
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    dx, dd, du = cr().cr_lora_backward(d["dY"], None, None, *tail, adapter=d["adapter"], base=d["dbase"],
                                       need_down=False, need_up=False)
    assert dd is None and du is None and torch.equal(dx, want[0])
    dx, dd, du = cr().cr_lora_backward(d["dY"], d["X"], None, *tail, adapter=d["adapter"], need_dx=False, need_up=False)
    assert dx is None and du is None and torch.equal(dd, want[1])
    dx, dd, du = cr().cr_lora_backward(d["dY"], None, V, *tail, adapter=d["adapter"], need_dx=False, need_down=False)
    assert dx is None and dd is None and torch.equal(du, want[2])


def test_no_rows():
    d = make(0, 512, 264, 8, 2, "all", seed=6)
    Y, V = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], base=d["base"], save_v=True)
    assert Y.shape == (0, 264) and V.shape == (0, 8)
    dX, dd, du = cr().cr_lora_backward(d["dY"], d["X"], V, d["down"], d["up"], d["scale"])
    assert dX.shape == (0, 512) and not dd.any() and not du.any()
    c, s = cr().cr_ckpt_save(d["X"])
    assert cr().cr_ckpt_load(c, s).shape == (0, 512)


@pytest.mark.parametrize("which", ["X", "down", "up"])
def test_gradients_against_differences(which):
    """The output is linear in each of X, down and up, so a difference over a whole step is exact up to the
    outputs' rounding: <dY, Y(t + d) - Y(t)> = <grad, d>, off by at most 2^-8 sum |dY| (|Y(t + d)| + |Y(t)|)
    and the gradient's own rounding, 2^-8 sum |grad d|."""
    d = make(96, 256, 128, 8, 2, "rows", seed=7)
    d["up"] *= 4
    kw = dict(adapter=d["adapter"])
    Y, V = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], save_v=True, **kw)
    dY = (Y.float() * 0.01).to(BF)  # a loss that pulls the output to zero
    grads = dict(zip(("X", "down", "up"), cr().cr_lora_backward(dY, d["X"], V, d["down"], d["up"], d["scale"], **kw)))
    step = grads[which].float()
    step = (step * (f64(d[which]).std() / f64(grads[which]).std())).to(BF)
    moved = dict(d)
    moved[which] = (d[which].float() + step.float()).to(BF)
    step = f64(moved[which]) - f64(d[which])
    Y2 = cr().cr_lora_forward(moved["X"], moved["down"], moved["up"], moved["scale"], **kw)
    diff = (f64(dY) * (f64(Y2) - f64(Y))).sum()
    along = (f64(grads[which]) * step).sum()
    # float32 sums add less than one more rounding of the outputs: twice the bound covers both
    tol = 2 * (ao.BF16 * (np.abs(f64(dY)) * (np.abs(f64(Y2)) + np.abs(f64(Y)))).sum()
               + ao.BF16 * np.abs(f64(grads[which]) * step).sum())
    assert along > 4 * tol  # the comparison says something
    assert abs(diff - along) <= tol


# ---------------------------------------------------------------------------------------------- checkpoints

def loud(g, M, K):
    x = torch.randn(M, K, device="cuda", generator=g)
    x[:, torch.rand(K, device="cuda", generator=g) < 0.02] *= 50
    return x.to(BF)


@pytest.mark.parametrize("M,K,pad", [(1, 256, 0), (7, 256, 8), (21, 2560, 0), (33, 768, 264), (130, 9728, 0), (1000, 1024, 0)])
def test_checkpoint(M, K, pad):
    x = loud(gen(M), M, K)
    codes, scales = cr().cr_ckpt_save(strided(x, pad))
    want, s, t = ao.ckpt_save(f64(x))
    got_s = scales.cpu().numpy()
    # float32 sums of 256 products with +-1, then an exact 1/16
    err = ao.steps(256) * np.abs(f64(x)).reshape(M, -1, 256).sum(-1) / 16
    assert (np.abs(got_s.astype(np.float64) - s) <= err / 127 + 2.0 ** -24 * s).all()
    c = codes.cpu().numpy().astype(np.int32)
    # a code may differ where y / s lies as near to a border as those roundings (and the scale's own) reach
    reach = np.repeat((2 * err / s + 127 * 2.0 ** -23), 256, axis=1).reshape(M, K)
    flips = c != want
    assert (np.abs(c - want) <= 1).all() and (np.abs(np.abs(t - np.floor(t)) - 0.5) <= reach)[flips].all()
    assert np.abs(c).max() <= 127
    # what the codes stand for: one float32 product and one rounding
    back, mags = ao.ckpt_values(codes.cpu().numpy(), got_s)
    out = torch.full((M, K + pad), float("nan"), dtype=BF, device="cuda")
    r = cr().cr_ckpt_load(codes, scales, out=out[:, :K])
    within(r, back, ao.BF16 * np.abs(back) + 2.0 ** -23 * np.abs(back) + 1e-300 * mags, "restored")
    assert torch.isnan(out[:, K:]).all()
    # half a step in every rotated value: at most sqrt(256) s / 2 = 8 s over a slice's norm
    d = (f64(r) - f64(x)).reshape(M, -1, 256)
    room = 8 * got_s + ao.BF16 * np.linalg.norm(back.reshape(M, -1, 256), axis=-1) + 16 * err
    assert (np.linalg.norm(d, axis=-1) <= room * (1 + 1e-6)).all()


def test_checkpoint_extremes():
    x = torch.zeros(6, 512, dtype=BF, device="cuda")
    x[1, 3] = 1e-38  # scale at its floor: comes back as zero
    x[2, 300] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 3e38  # the rotation leaves float32
    x[5, :256] = 2.0 ** 100
    c, s = cr().cr_ckpt_save(x)
    r = cr().cr_ckpt_load(c, s)
    assert not r[:2].any() and not c[:2].any()
    assert torch.isnan(r[2, 256:]).all() and not r[2, :256].any() and not c[2].any()
    assert torch.isnan(r[3, :256]).all() and not r[3, 256:].any()
    assert torch.isnan(r[4]).all()
    assert torch.isfinite(r[5]).all() and float((r[5, :256].double() / 2.0 ** 100 - 1).abs().max()) <= 2.0 ** -7 + 8 / 127


def test_checkpoint_past_32_bit_offsets():
    M, K = 40000, 65536  # 2.6e9 values
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[-1] = loud(gen(1), 1, K)[0]
    c, s = cr().cr_ckpt_save(x)
    assert not c[:-1].any()
    c1, s1 = cr().cr_ckpt_save(x[-1:].contiguous())
    assert torch.equal(c[-1:], c1) and torch.equal(s[-1:], s1)
    x.fill_(1)
    r = cr().cr_ckpt_load(c, s, out=x)
    assert not r[:-1].any() and torch.equal(r[-1:], cr().cr_ckpt_load(c1, s1))


# ---------------------------------------------------------------------------------------------- input gradient

@pytest.mark.parametrize("M,K,N,group,mode", [
    (1, 256, 8, 256, "tensor"), (1, 2560, 9728, 256, "row"), (21, 1024, 136, 1024, "row"), (130, 512, 256, 16, "tensor"),
    (129, 768, 264, 64, "row"), (257, 1280, 1000, 256, "tensor"), (300, 9728, 2560, 256, "row"), (1030, 3072, 1544, 256, "tensor"),
    (5, 4096, 72, 1024, "tensor"), (64, 512, 64, 64, "row"), (128, 1024, 520, 16, "row"), (512, 512, 320, 256, "tensor"),
    (513, 512, 320, 256, "row"), (300, 256, 520, 64, "row"), (512, 256, 1024, 256, "tensor"), (600, 2048, 200, 1024, "tensor"), (77, 256, 2048, 256, "row"),
    # straight from the packed weights: enough of them for each token
    (3, 512, 520, 16, "row"), (130, 2048, 2304, 64, "row"), (200, 2048, 4008, 1024, "row"), (257, 4096, 2312, 256, "tensor"),
    (600, 4096, 5128, 256, "row"), (512, 5120, 3600, 16, "tensor")])
def test_grad_input(M, K, N, group, mode):
    g = gen(M + N)
    W = randn(g, N, K, std=0.02)
    Wq, s = cr().cr_pack_weight(W, group=group, scale_mode=mode)
    dY = randn(g, M, N, std=1e-3)
    want, bound = ao.grad_input(f64(dY), Wq.cpu().numpy(), s.cpu().numpy(), group)
    within(cr().cr_w4a4_grad_input(dY, Wq, s, group=group), want, bound, "dX")
    out = torch.full((M, K + 8), float("nan"), dtype=BF, device="cuda")
    within(cr().cr_w4a4_grad_input(strided(dY, 32), Wq, s, group=group, out=out[:, :K]), want, bound, "dX, strided")
    assert torch.isnan(out[:, K:]).all()


def test_grad_input_empty():
    dY = torch.zeros(4, 0, dtype=BF, device="cuda")
    Wq, s = torch.zeros(0, 128, dtype=torch.uint8, device="cuda"), torch.zeros(0, device="cuda")
    assert not cr().cr_w4a4_grad_input(dY, Wq, s).any()
    dY = torch.zeros(0, 8, dtype=BF, device="cuda")
    Wq, s = torch.zeros(8, 128, dtype=torch.uint8, device="cuda"), torch.zeros(8, device="cuda")
    assert cr().cr_w4a4_grad_input(dY, Wq, s).shape == (0, 256)


def test_grad_input_keeps_non_finite_rows_apart():
    g = gen(9)
    Wq, s = cr().cr_pack_weight(randn(g, 264, 512))
    dY = randn(g, 200, 264)
    want = cr().cr_w4a4_grad_input(dY, Wq, s)
    dY[77, 5] = float("nan")
    got = cr().cr_w4a4_grad_input(dY, Wq, s)
    ok = torch.arange(200, device="cuda") != 77
    assert torch.equal(got[ok], want[ok]) and torch.isnan(got[77]).all()


# ---------------------------------------------------------------------------------------------- together

def step(d, Wq, s_w):
    """One training step's calls around a frozen packed layer with adapters, as a user makes them."""
    m = cr()
    kept = m.cr_ckpt_save(d["X"])
    y0 = m.cr_w4a4_linear(d["X"], Wq, s_w)
    Y, V = m.cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], base=y0, out=y0, save_v=True)
    dx0 = m.cr_w4a4_grad_input(d["dY"], Wq, s_w)
    dX, dd, du = m.cr_lora_backward(d["dY"], kept, V, d["down"], d["up"], d["scale"], adapter=d["adapter"], base=dx0,
                                    out=dx0)
    return Y, dX, dd, du


@pytest.mark.parametrize("M,mix", [(40, "rows"), (700, "runs")])
def test_training_step(M, mix):
    d = make(M, 512, 768, 16, 3, mix, seed=11)
    Wq, s_w = cr().cr_pack_weight(randn(gen(12), 768, 512, std=0.02))
    Y, dX, dd, du = step(d, Wq, s_w)
    torch.cuda.synchronize()
    down, up, sc, a = f64(d["down"]), f64(d["up"]), f64(d["scale"]), ids(d["adapter"])
    y0 = f64(cr().cr_w4a4_linear(d["X"], Wq, s_w))
    want, v, ey, _ = ao.lora_forward(f64(d["X"]), down, up, sc, a, y0)
    within(Y, want, ey, "Y")
    dx0, e0 = ao.grad_input(f64(d["dY"]), Wq.cpu().numpy(), s_w.cpu().numpy())
    codes, scales = cr().cr_ckpt_save(d["X"])
    x, mags = ao.ckpt_values(codes.cpu().numpy(), scales.cpu().numpy())
    V = torch.from_numpy(v).to(BF).double().numpy()  # may differ by a step from the kernel's
    (wx, wd, wu), (ex, ed, eu) = ao.lora_backward(f64(d["dY"]), x, V, down, up, sc, a, dx0, mags)
    within(dX, wx, ex + e0 * (1 + ao.BF16), "dX")
    within(dd, wd, ed, "d_down")
    extra = np.stack([sc[k] * 2 * ao.BF16 * (np.abs(v[r]).T @ np.abs(f64(d["dY"])[r])) for k, r in ao.row_masks(a, M, 3)])
    within(du, wu, eu + extra, "d_up")


def test_other_stream_and_captured_graphs():
    """Two captured steps of different sizes replayed in turn and together with eager calls on another
    stream: every result as the eager call's."""
    Wq, s_w = cr().cr_pack_weight(randn(gen(12), 768, 512, std=0.02))
    sets = [make(700, 512, 768, 16, 3, "runs", seed=21), make(60, 512, 768, 64, 5, "rows", seed=22)]
    want = [[t.clone() for t in step(d, Wq, s_w)] for d in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in sets:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(d, Wq, s_w)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(d, Wq, s_w))
        graphs.append(g)
    for o in outs:
        for t in o:
            t.fill_(float("nan"))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        for g in graphs:
            g.replay()
        with torch.cuda.stream(other):
            eager = cr().cr_lora_forward(sets[0]["X"], sets[0]["down"], sets[0]["up"], sets[0]["scale"],
                                         adapter=sets[0]["adapter"])
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for x, y in zip(o, w):
                assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    ref = cr().cr_lora_forward(sets[0]["X"], sets[0]["down"], sets[0]["up"], sets[0]["scale"], adapter=sets[0]["adapter"])
    assert torch.equal(eager, ref)


def test_own_workspace_and_status():
    d = make(3000, 512, 264, 16, 2, "runs", seed=31)
    from w4a8_rotated_quantized_b200 import binding

    n = binding._lib.cr_lora_forward_workspace_size(3000, 264, 512, 16, 2)
    assert binding._lib.cr_lora_forward_workspace_size(3, 264, 512, 16, 2) == 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # nothing needs to be zero before
    want = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"])
    got = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], workspace=ws)
    assert torch.equal(got, want) and cr().cr_read_device_status(ws=ws) == 0
    with pytest.raises(cr().ConvRotError):
        cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], workspace=ws[:256])
    ws.fill_(255)  # few rows: needs none, and says so in one that it is given
    few = cr().cr_lora_forward(d["X"][:3], d["down"], d["up"], d["scale"], adapter=d["adapter"][:3], workspace=ws[:256])
    assert torch.isfinite(few).all() and cr().cr_read_device_status(ws=ws) == 0


def test_refusals():
    m = cr()
    d = make(8, 512, 264, 8, 2, "rows", seed=41)
    ok = (d["X"], d["down"], d["up"], d["scale"])
    with pytest.raises(TypeError):
        m.cr_lora_forward(d["X"].float(), *ok[1:])
    with pytest.raises(ValueError):
        m.cr_lora_forward(d["X"][:, :256], *ok[1:])  # K disagrees with down
    with pytest.raises(TypeError):
        m.cr_lora_forward(*ok, adapter=d["adapter"].long())
    with pytest.raises(ValueError):
        m.cr_lora_forward(*ok, adapter=d["adapter"][:-1])
    with pytest.raises(ValueError):
        m.cr_lora_forward(*ok, base=d["base"][:4])
    with pytest.raises(m.ConvRotError):
        m.cr_lora_forward(*ok, base=d["base"][:1].expand(8, 264))  # rows that lie on one another
    with pytest.raises(m.ConvRotError):
        m.cr_lora_forward(d["X"], d["down"][:, :6].contiguous(), d["up"][:, :6].contiguous(), d["scale"])  # rank % 4
    with pytest.raises(ValueError):
        m.cr_lora_backward(d["dY"], None, None, *ok[1:], need_up=False)
    with pytest.raises(ValueError):
        m.cr_lora_backward(d["dY"], (torch.zeros(8, 512, dtype=torch.int8, device="cuda"), torch.zeros(8, 1, device="cuda")),
                           None, *ok[1:], need_up=False)
    with pytest.raises(m.ConvRotError):
        m.cr_ckpt_save(d["X"][:, :264].contiguous())  # K % 256
    with pytest.raises(m.ConvRotError):
        m.cr_w4a4_grad_input(d["base"], torch.zeros(264, 256, dtype=torch.uint8, device="cuda"),
                             torch.ones(264, device="cuda"), group=32)


# ---------------------------------------------------------------------------------------------- many times, large, side by side

@pytest.mark.parametrize("M,K,N,r,L,mix,kept", [(8192, 2048, 512, 32, 1, "all", "int8"), (1500, 512, 1024, 128, 1, "all", "bf16"),
                                                (1500, 512, 1024, 128, 3, "runs", "bf16"), (3000, 256, 256, 80, 2, "rows", "int8"),
                                                (700, 1024, 256, 12, 6, "rows", "bf16")])
def test_the_same_bits_a_hundred_times(M, K, N, r, L, mix, kept):
    """Waits that are answered too early show as rare differences."""
    d = make(M, K, N, r, L, mix, seed=51)
    Wq, s_w = cr().cr_pack_weight(randn(gen(52), N, K, std=0.02))

    def once():
        Y, V = cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], base=d["base"], save_v=True)
        keep = cr().cr_ckpt_save(d["X"])
        g = cr().cr_lora_backward(d["dY"], keep if kept == "int8" else d["X"], V, d["down"], d["up"], d["scale"],
                                  adapter=d["adapter"], base=d["dbase"])
        return (Y, V, *keep, *g, cr().cr_w4a4_grad_input(d["dY"], Wq, s_w), cr().cr_w4a4_grad_input(d["dY"][:200], Wq, s_w))

    want = once()
    wrong = torch.zeros(len(want), device="cuda")
    for _ in range(100):
        wrong += torch.stack([(a.view(torch.uint8) != b.view(torch.uint8)).any() for a, b in zip(once(), want)])
    assert not wrong.any(), wrong.tolist()


def test_two_streams_at_once():
    sets = [make(900, 512, 768, 16, 3, "runs", seed=61), make(50, 1024, 512, 64, 4, "rows", seed=62)]
    want = [cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], base=d["base"]) for d in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, d in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], base=d["base"]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_adapters_past_32_bit_offsets():
    """270000 x 8192 values: only the last rows name an adapter, and all others pass through."""
    M, K, N, r = 270000, 8192, 64, 8
    g = gen(71)
    X = torch.zeros(M, K, dtype=BF, device="cuda")
    X[-3:] = randn(g, 3, K)
    a = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    a[-3:] = torch.tensor([1, 0, 1], dtype=torch.int32)
    down, up = randn(g, 2, r, K, std=K ** -0.5), randn(g, 2, r, N)
    scale = torch.tensor([0.5, 2.0], device="cuda")
    Y, V = cr().cr_lora_forward(X, down, up, scale, adapter=a, save_v=True)
    Y3, V3 = cr().cr_lora_forward(X[-3:], down, up, scale, adapter=a[-3:], save_v=True)
    want, v, ey, ev = ao.lora_forward(f64(X[-3:]), f64(down), f64(up), f64(scale), ids(a[-3:]))
    for got, w, e in ((Y[-3:], want, ey), (Y3, want, ey), (V[-3:], v, ev), (V3, v, ev)):
        within(got, w, e, "last rows")
    assert not Y[:-3].any() and not V[:-3].any()
    # and the other way round: wide outputs, gradients of the wide side
    dY = torch.zeros(M, N, dtype=BF, device="cuda")
    dY[-3:] = randn(g, 3, N)
    dX, dd, du = cr().cr_lora_backward(dY, X, V, down, up, scale, adapter=a)
    (wx, wd, wu), (ex, ed, eu) = ao.lora_backward(f64(dY[-3:]), f64(X[-3:]), f64(V[-3:]), f64(down), f64(up), f64(scale), ids(a[-3:]))
    within(dX[-3:], wx, ex, "dX")
    within(dd, wd, ed, "d_down")
    within(du, wu, eu, "d_up")
    assert not dX[:-3].any()
    del dX
    kept = cr().cr_ckpt_save(X)
    x, mags = ao.ckpt_values(kept[0][-3:].cpu().numpy(), kept[1][-3:].cpu().numpy())
    (_, wd, _), (_, ed, _) = ao.lora_backward(f64(dY[-3:]), x, f64(V[-3:]), f64(down), f64(up), f64(scale), ids(a[-3:]), None, mags)
    within(cr().cr_lora_backward(dY, kept, V, down, up, scale, adapter=a, need_dx=False, need_up=False)[1], wd, ed, "d_down from codes")


def test_grad_input_past_32_bit_offsets():
    M, K, N = 140000, 256, 16384
    g = gen(72)
    dY = torch.zeros(M, N, dtype=BF, device="cuda")
    dY[-2:] = randn(g, 2, N)
    Wq, s = cr().cr_pack_weight(randn(g, N, K, std=0.02), scale_mode="row")
    want, bound = ao.grad_input(f64(dY[-2:]), Wq.cpu().numpy(), s.cpu().numpy())
    got = cr().cr_w4a4_grad_input(dY, Wq, s)
    within(got[-2:], want, bound, "dX")
    assert not got[:-2].any()


def test_views_at_odd_places():
    """Row indices, scales and V that start anywhere their elements may."""
    d = make(260, 512, 264, 4, 3, "rows", seed=81)
    a = torch.zeros(261, dtype=torch.int32, device="cuda")
    a[1:] = d["adapter"]
    sc = torch.zeros(4, device="cuda")
    sc[1:] = d["scale"]
    args = (d["X"], d["down"], d["up"])
    Y, V = cr().cr_lora_forward(*args, d["scale"], adapter=d["adapter"], base=d["base"], save_v=True)
    Y2, V2 = cr().cr_lora_forward(*args, sc[1:], adapter=a[1:], base=d["base"], save_v=True)
    assert torch.equal(Y, Y2) and torch.equal(V, V2)
    rows = slice(1, 260)  # every operand one row further: V's rows are 8 bytes long
    g = cr().cr_lora_backward(d["dY"][rows], d["X"][rows], V[rows], d["down"], d["up"], sc[1:], adapter=a[1:][rows])
    want, bound = ao.lora_backward(f64(d["dY"][rows]), f64(d["X"][rows]), f64(V[rows]), f64(d["down"]), f64(d["up"]),
                                   f64(d["scale"]), ids(d["adapter"][rows]))
    for x, w, b, name in zip(g, want, bound, ("dX", "d_down", "d_up")):
        within(x, w, b, name)


def test_output_on_another_operand_is_refused():
    d = make(40, 256, 256, 8, 2, "rows", seed=91)
    with pytest.raises(cr().ConvRotError):
        cr().cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], out=d["X"])
    with pytest.raises(cr().ConvRotError):
        cr().cr_lora_backward(d["dY"], d["X"], None, d["down"], d["up"], d["scale"], out=d["X"], need_up=False)
    Wq, s = cr().cr_pack_weight(randn(gen(92), 256, 256))
    with pytest.raises(cr().ConvRotError):
        cr().cr_w4a4_grad_input(d["dY"], Wq, s, out=d["dY"])


@pytest.mark.parametrize("M,L,mix", [(1, 1, "all"), (3, 4, "rows"), (60, 3, "runs"), (300, 2, "runs"), (700, 9, "rows")])
def test_calls_on_each_others_results(M, L, mix):
    """Calls whose kernels start beside the end of the call before, each reading or overwriting what that one
    wrote or read, with nothing else between them: the same bits as with a synchronisation after every call."""
    m = cr()
    d = make(M, 512, 512, 16, L, mix, seed=71)
    Wq, s_w = m.cr_pack_weight(randn(gen(72), 512, 512, std=0.04))
    scale, a = d["scale"] * 0.1, d["adapter"]

    def run(between):
        A, B, seen = d["X"].clone(), d["base"].clone(), []
        torch.cuda.synchronize()
        for _ in range(8):
            _, V = m.cr_lora_forward(A, d["down"], d["up"], scale, adapter=a, base=B, out=B, save_v=True)
            between()
            codes, scales = m.cr_ckpt_save(A)
            between()
            m.cr_ckpt_load(codes, scales, out=A)
            between()
            _, dd, du = m.cr_lora_backward(B, (codes, scales), V, d["down"], d["up"], scale, adapter=a, base=A, out=A)
            between()
            Y = m.cr_lora_forward(B, dd, du, scale, adapter=a, base=A)
            between()
            m.cr_w4a4_grad_input(A, Wq, s_w, out=B)
            between()
            _, dd2, _ = m.cr_lora_backward(B, A, None, dd, du, scale, adapter=a, need_dx=False, need_up=False)
            between()
            seen += [Y, dd, du, dd2]
        torch.cuda.synchronize()
        return seen + [A, B]

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        got = run(lambda: None)
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(got, want))


def test_after_other_work_on_the_stream():
    """Calls behind a copy, a memset, another stream's event and each other, eagerly and captured: their kernels
    start beside the end of what is before them and must not read too early."""
    m = cr()
    sets = [make(3, 512, 768, 16, 3, "rows", seed=81), make(300, 512, 768, 64, 2, "runs", seed=82)]
    Wq, s_w = m.cr_pack_weight(randn(gen(83), 768, 512, std=0.02))
    side = torch.cuda.Stream()
    late = [{k: torch.zeros_like(v) if torch.is_tensor(v) else v for k, v in d.items()} for d in sets]
    slow = torch.zeros(64 << 20, device="cuda")

    def calls(i):
        here, d, t = torch.cuda.current_stream(), sets[i], late[i]
        for k in d:  # whatever the call before left there goes
            if torch.is_tensor(d[k]):
                t[k].zero_()
        for k in ("down", "up", "scale", "adapter", "base"):  # copies right before the call
            t[k].copy_(d[k])
        side.wait_stream(here)
        with torch.cuda.stream(side):  # and rows from another stream, after something long
            slow.add_(1)
            t["X"].copy_(d["X"])
            t["dY"].copy_(d["dY"])
        here.wait_stream(side)
        Y, V = m.cr_lora_forward(t["X"], t["down"], t["up"], t["scale"], adapter=t["adapter"], base=t["base"], save_v=True)
        t["X"].zero_()
        t["X"].copy_(d["X"])
        kept = m.cr_ckpt_save(t["X"])
        back = m.cr_ckpt_load(*kept)
        _, _, du = m.cr_lora_backward(t["dY"], None, V, t["down"], t["up"], t["scale"], adapter=t["adapter"],
                                      need_dx=False, need_down=False)
        g = m.cr_lora_backward(t["dY"], kept, V, t["down"], t["up"], t["scale"], adapter=t["adapter"])
        t["dY"].zero_()
        t["dY"].copy_(d["dY"])
        return (Y, V, *kept, back, du, *g, m.cr_w4a4_grad_input(t["dY"], Wq, s_w))

    def same(a, b):
        return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))

    for i, d in enumerate(sets):
        Y, V = m.cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=d["adapter"], base=d["base"], save_v=True)
        torch.cuda.synchronize()
        kept = m.cr_ckpt_save(d["X"])
        torch.cuda.synchronize()
        back = m.cr_ckpt_load(*kept)
        g = m.cr_lora_backward(d["dY"], kept, V, d["down"], d["up"], d["scale"], adapter=d["adapter"])
        torch.cuda.synchronize()
        want = (Y, V, *kept, back, g[2], *g, m.cr_w4a4_grad_input(d["dY"], Wq, s_w))
        torch.cuda.synchronize()
        for _ in range(3):
            assert same(calls(i), want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls(i)
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert same(got, want)


@pytest.mark.parametrize("M,kept", [(2, "bf16"), (300, "int8"), (2600, "bf16"), (2600, "int8")])
def test_no_indices_and_a_pool_of_several(M, kept):
    """Without indices every row has the pool's first adapter; the others' gradients are zero."""
    m = cr()
    d = make(M, 512, 776, 40, 3, "all", seed=91)
    zeros = torch.zeros(M, dtype=torch.int32, device="cuda")
    X = m.cr_ckpt_save(d["X"]) if kept == "int8" else d["X"]
    got = []
    for a in (None, zeros):
        Y, V = m.cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], adapter=a, base=d["base"], save_v=True)
        got.append((Y, V, *m.cr_lora_backward(d["dY"], X, V, d["down"], d["up"], d["scale"], adapter=a, base=d["dbase"])))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert not got[0][3][1:].any() and not got[0][4][1:].any() and got[0][3][0].any() and got[0][4][0].any()


@pytest.mark.parametrize("M", [3, 40, 600])
def test_indices_and_scales_written_right_before_a_call(M):
    """Every call meets indices and scales that are not those of the call before, written by the work right in front
    of it: by a copy, or by checkpoints saved into them (a kernel that lets the call start beside its end).  The same
    bits as with a synchronisation after every piece."""
    m = cr()
    from w4a8_rotated_quantized_b200 import binding

    K = N = 512
    L, rounds = 4, 6
    d = make(M, K, N, 16, L, "all", seed=101)
    g = gen(102)
    Wq, _ = m.cr_pack_weight(randn(g, N, K, std=0.04))
    _, V = m.cr_lora_forward(d["X"], d["down"], d["up"], d["scale"], save_v=True)

    # Rows whose rotated values are, four bytes to an index: an index of -0 .. L (L: none) in the lowest, zeros in the
    # others, and 127 in the last index of each row, which makes the scale 1 and is no adapter.
    rows = (M + 63) // 64
    want_ids = torch.randint(0, L + 1, (rounds, rows, 64), device="cuda", generator=g, dtype=torch.int32)
    want_ids[:, :, 63] = 127
    y = torch.zeros(rounds, rows, 64, 4, device="cuda", dtype=torch.float64)
    y[..., 0] = want_ids.double()
    h = torch.from_numpy(np.asarray(oracle.regular_hadamard(256), np.float64)).cuda()
    id_rows = (y.reshape(rounds, rows, 256) @ h).to(BF)
    scale_rows = randn(g, rounds, L, 256)  # scales of about 0.02, all different
    w_rows = randn(g, rounds, N, 256)

    codes = torch.zeros(max(rows, N), 256, dtype=torch.int8, device="cuda")
    adapter = codes.view(torch.int32).reshape(-1)[:M]
    spare = torch.zeros(max(rows, N), 256, dtype=torch.int8, device="cuda")
    one = torch.zeros(rows, device="cuda")
    scale, w_scale = torch.zeros(L, device="cuda"), torch.zeros(N, device="cuda")
    ptr = binding._ptr

    def save(x, codes, scales):
        binding._check("cr_ckpt_save", binding._lib.cr_ckpt_save(ptr(x), x.shape[0], 256, 256, ptr(codes), ptr(scales),
                                                                 binding._stream(x.device)))

    def run(between):
        codes.zero_(), scale.zero_(), w_scale.zero_()
        torch.cuda.synchronize()
        seen = []
        calls = (lambda: m.cr_lora_forward(d["X"], d["down"], d["up"], scale, adapter=adapter, base=d["base"], save_v=True),
                 lambda: m.cr_lora_backward(d["dY"], d["X"], V, d["down"], d["up"], scale, adapter=adapter, base=d["dbase"]),
                 lambda: m.cr_lora_backward(d["dY"], None, V, d["down"], d["up"], scale, adapter=adapter, need_dx=False,
                                            need_down=False)[2:])
        for k in range(rounds):
            for i, call in enumerate(calls):
                j = (k + i) % rounds
                save(scale_rows[j], spare, scale)
                between()
                save(id_rows[j], codes, one)
                between()
                seen += [*call(), adapter.clone()]
                between()
                save(id_rows[(j + 1) % rounds], codes, one)
                between()
                save(scale_rows[(j + 1) % rounds], spare, scale)
                between()
                seen += call()
                between()
                adapter.copy_(want_ids[j].reshape(-1)[:M])
                between()
                scale.copy_(one[:1].expand(L) * (j + 1))
                between()
                seen += call()
                between()
            save(w_rows[k], spare, w_scale)
            between()
            seen.append(m.cr_w4a4_grad_input(d["dY"], Wq, w_scale))
            between()
            w_scale.copy_(w_scale.flip(0))
            between()
            seen.append(m.cr_w4a4_grad_input(d["dY"], Wq, w_scale))
            between()
        torch.cuda.synchronize()
        return seen

    want = run(torch.cuda.synchronize)
    assert torch.equal(want[2], want_ids[0].reshape(-1)[:M])  # the checkpoint's codes are the indices meant
    for _ in range(5):
        got = run(lambda: None)
        for x, w in zip(got, want):
            assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))


def test_empty_calls_write_the_status_word():
    """A call without rows, or without anything to make, says so in the workspace that it is given, too."""
    m = cr()
    d = make(0, 512, 264, 8, 2, "all", seed=111)
    full = make(5, 512, 264, 8, 2, "rows", seed=112)
    tail = (d["down"], d["up"], d["scale"])
    codes = torch.zeros(0, 512, dtype=torch.int8, device="cuda"), torch.zeros(0, 2, device="cuda")
    V = torch.zeros(0, 8, dtype=BF, device="cuda")
    Wq, s = m.cr_pack_weight(randn(gen(113), 264, 512))
    none = torch.zeros(5, 0, dtype=BF, device="cuda")
    from w4a8_rotated_quantized_b200 import binding

    size = max(binding._lib.cr_lora_backward_workspace_size(M, 264, 512, 8, 2) for M in (0, 5))
    size = max(size, binding._lib.cr_w4a4_grad_input_workspace_size(0, 264, 512, 256))
    for call in (lambda ws: m.cr_lora_forward(d["X"], *tail, base=d["base"], workspace=ws),
                 lambda ws: m.cr_lora_backward(d["dY"], d["X"], V, *tail, workspace=ws),
                 lambda ws: m.cr_lora_backward(d["dY"], codes, V, *tail, workspace=ws),
                 lambda ws: m.cr_lora_backward(full["dY"], None, None, *tail, need_dx=False, need_down=False, need_up=False,
                                               workspace=ws),
                 lambda ws: m.cr_w4a4_grad_input(d["dY"], Wq, s, workspace=ws),
                 lambda ws: m.cr_w4a4_grad_input(none, Wq[:0], s[:0], workspace=ws)):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        call(ws)
        assert m.cr_read_device_status(ws=ws) == 0
        assert not ws[:16].any() and (ws[16:] == 255).all()  # and nothing else


@pytest.mark.parametrize("r", [8, 64])
@pytest.mark.parametrize("M", [3, 600])
def test_infinities_by_the_formula(M, r):
    """An infinite V or dV gives infinities of the formula's sign and a V past bf16's largest value finite results,
    in the form for few rows and in the one for batches, of up to 32 ranks and of more."""
    m = cr()
    K, N, inf = 64, 72, float("inf")
    X = torch.zeros(M, K, dtype=BF, device="cuda")
    X[:, 0] = 1
    X[0, 1] = inf  # V infinite
    X[1, 1] = float("nan")
    # 2^128 - 2^120 is bf16's largest value; with 1.5 * 2^119 more V is float32 still, but rounds to an infinity
    X[2, 0], X[2, 2] = 2.0 ** 128 - 2.0 ** 120, 1.5 * 2.0 ** 119
    down = torch.zeros(2, r, K, dtype=BF, device="cuda")
    down[:, 0, :3] = 1
    down[:, 1:, 0] = 2.0 ** -126
    down[:, 1:, 1] = 1
    up = torch.full((2, r, N), 2.0 ** -30, dtype=BF, device="cuda")
    up[:, :, 1::2] *= -1
    scale = torch.tensor([1.0, inf], device="cuda")
    a = torch.zeros(M, dtype=torch.int32, device="cuda")
    if M > 3:
        a[3] = 1  # scale infinite
    Y, V = m.cr_lora_forward(X, down, up, scale, adapter=a, save_v=True)
    sign = torch.ones(N, device="cuda")
    sign[1::2] = -1
    assert (V[0] == inf).all() and torch.isnan(V[1]).all() and V[2, 0] == inf and torch.isfinite(V[2, 1:]).all()
    assert torch.equal(Y[0].float(), sign * inf) and torch.isnan(Y[1]).all()
    v, want = f64(X[2]) @ f64(down[0]).T, f64(up[0])
    want = v @ want
    # one rounding of the output, the pair's 2^-16, float32 sums of r products
    within(Y[2], want, np.abs(want) * (ao.BF16 + ao.PAIR + ao.steps(2 * r)), "Y")
    assert torch.isfinite(Y[4:]).all()
    if M > 3:
        assert torch.equal(Y[3].float(), sign * inf)
    # backward: dV of row 0 infinite, X positive in one column and negative in another, one row to an adapter
    dY = torch.zeros(M, N, dtype=BF, device="cuda")
    dY[0, 0], dY[1:, 0] = inf, 1
    a = torch.full((M,), 1, dtype=torch.int32, device="cuda")
    a[0] = 0
    Z = torch.ones(M, K, dtype=BF, device="cuda")
    Z[:, 1::2] = -1
    flip = torch.ones(K, device="cuda")
    flip[1::2] = -1
    down = torch.ones(2, r, K, dtype=BF, device="cuda")
    down[:, :, 1::2] = -1
    dX, dd, _ = m.cr_lora_backward(dY, Z, None, down, up, torch.ones(2, device="cuda"), adapter=a, need_up=False)
    assert torch.equal(dX[0].float(), flip * inf) and torch.isfinite(dX[1:]).all()
    assert torch.equal(dd[0].float(), (flip * inf).expand(r, K)) and torch.isfinite(dd[1]).all()


@pytest.mark.parametrize("M", [4, 300])
def test_copy_on_write_outputs_are_made_their_own(M):
    """An output that shares its memory with another tensor until it is written: the other keeps its values."""
    m = cr()
    d = make(M, 512, 512, 8, 2, "rows", seed=121)
    tail, a = (d["down"], d["up"], d["scale"]), d["adapter"]
    Wq, s = m.cr_pack_weight(randn(gen(122), 512, 512))
    kept = m.cr_ckpt_save(d["X"])
    for shared, call in ((d["base"], lambda **k: m.cr_lora_forward(d["X"], *tail, adapter=a, **k)),
                         (d["dbase"], lambda **k: m.cr_lora_backward(d["dY"], None, None, *tail, adapter=a, need_down=False,
                                                                     need_up=False, **k)[0]),
                         (d["X"], lambda **k: m.cr_ckpt_load(*kept, **k)),
                         (d["dY"], lambda **k: m.cr_w4a4_grad_input(d["dY"], Wq, s, **k))):
        before = shared.clone()
        for in_place in (False, True) if shared is d["base"] or shared is d["dbase"] else (False,):
            want = call(**({"base": shared} if in_place else {}))
            out = torch._lazy_clone(shared)
            got = call(out=out, **({"base": out} if in_place else {}))
            assert got is out and torch.equal(out, want) and torch.equal(shared, before)
            assert out.data_ptr() != shared.data_ptr()


@pytest.mark.parametrize("group", [(1 << 32) + 256, -(1 << 32) + 64, 1 << 31, 1 << 80])
def test_a_group_past_32_bits_is_refused(group):
    m = cr()
    Wq, s = m.cr_pack_weight(randn(gen(131), 8, 256))
    with pytest.raises((ValueError, OverflowError)):
        m.cr_w4a4_grad_input(randn(gen(132), 4, 8), Wq, s, group=group)


@pytest.mark.parametrize("power", [-90, 40, 100, 112])
def test_checkpoint_over_its_range(power):
    """A power of two on the values is one on the scales and leaves the codes, up to magnitudes that add up to
    almost 2^128 in a slice and down to scales of 2^-100."""
    m = cr()
    x = torch.randn(140, 768, device="cuda", generator=gen(141)).clamp(-4, 4)
    x *= 2.0 ** 15 / x.abs().reshape(140, 3, 256).sum(-1).max()  # at most 2^15 in all, before one rounding
    x = (x * 0.99).to(BF)
    assert x.abs().double().reshape(140, 3, 256).sum(-1).max() < 2.0 ** 15
    c, s = m.cr_ckpt_save(x)
    y = (x.double() * 2.0 ** power).to(BF)
    assert torch.equal(y.double(), x.double() * 2.0 ** power)  # exact
    c2, s2 = m.cr_ckpt_save(y)
    assert torch.equal(c, c2) and torch.equal(s2.double(), s.double() * 2.0 ** power)
    r, r2 = m.cr_ckpt_load(c, s), m.cr_ckpt_load(c2, s2)
    assert torch.isfinite(r2).all() and torch.equal(r2.double(), r.double() * 2.0 ** power)


@pytest.mark.parametrize("M,N", [(3, 2640), (600, 264)])
def test_weight_scales_at_odd_places(M, N):
    """Weight scales that start at any float: straight from the packed weights and by way of the unpacked ones."""
    m = cr()
    Wq, s = m.cr_pack_weight(randn(gen(151), N, 512, std=0.02), scale_mode="row")
    dY = randn(gen(152), M, N, std=1e-3)
    want = m.cr_w4a4_grad_input(dY, Wq, s)
    for off in (1, 2, 3):
        odd = torch.full((N + off + 1,), float("nan"), device="cuda")
        odd[off:off + N] = s
        assert torch.equal(m.cr_w4a4_grad_input(dY, Wq, odd[off:off + N]), want)
