"""Adapter, checkpoint and input-gradient calls without a GPU: the oracle against its definitions, the
ABI's refusals (fake device pointers, never dereferenced) and the binding's argument checks."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import adapter_oracle as ao
from w4a8_rotated_quantized_b200 import binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _case(seed=0, M=9, K=256, N=16, r=4, L=3):
    g = np.random.default_rng(seed)
    return dict(x=g.standard_normal((M, K)), down=g.standard_normal((L, r, K)), up=g.standard_normal((L, r, N)),
                scale=g.random(L), adapter=g.integers(-1, L + 1, M), base=g.standard_normal((M, N)),
                dy=g.standard_normal((M, N)))


def test_oracle_forward_row_by_row():
    c = _case()
    y, v, ey, ev = ao.lora_forward(**{k: c[k] for k in ("x", "down", "up", "scale", "adapter", "base")})
    for m, a in enumerate(c["adapter"]):
        if 0 <= a < 3:
            want = c["base"][m] + c["scale"][a] * (c["up"][a].T @ (c["down"][a] @ c["x"][m]))
        else:
            want = c["base"][m]
            assert not v[m].any()
        assert np.allclose(y[m], want, rtol=1e-12, atol=1e-12)
    assert (ey >= 0).all() and (ev >= 0).all()


@pytest.mark.parametrize("name", ["x", "down", "up"])
def test_oracle_gradients_against_differences(name):
    c = _case(1)
    keys = ("x", "down", "up", "scale", "adapter", "base")
    y, v, *_ = ao.lora_forward(**{k: c[k] for k in keys})
    (dx, dd, du), _ = ao.lora_backward(c["dy"], c["x"], v, c["down"], c["up"], c["scale"], c["adapter"])
    grad = {"x": dx, "down": dd, "up": du}[name]
    step = np.random.default_rng(2).standard_normal(grad.shape)
    y2, *_ = ao.lora_forward(**{**{k: c[k] for k in keys}, name: c[name] + step})
    assert np.isclose((c["dy"] * (y2 - y)).sum(), (grad * step).sum(), rtol=1e-10)


def test_oracle_checkpoint_round_trip():
    x = np.random.default_rng(3).standard_normal((5, 512)) * 3
    codes, s, _ = ao.ckpt_save(x)
    back, mags = ao.ckpt_values(codes, s)
    err = np.linalg.norm((back - x).reshape(5, 2, 256), axis=-1)
    assert (err <= 8 * s * (1 + 1e-6)).all() and np.abs(codes).max() == 127 and (mags >= np.abs(back) - 1e-12).all()
    h = ao.rotate64(np.eye(256))
    assert np.allclose(h @ h, np.eye(256)) and np.allclose(h, h.T)


def test_oracle_bound_catches_a_planted_mistake():
    c = _case(4)
    y, v, ey, _ = ao.lora_forward(**{k: c[k] for k in ("x", "down", "up", "scale", "adapter", "base")})
    bad = c["down"].copy()
    bad[1, 2] = 0  # one rank row of one adapter lost
    y2, *_ = ao.lora_forward(c["x"], bad, c["up"], c["scale"], c["adapter"], c["base"])
    hit = c["adapter"] == 1
    assert hit.any() and (np.abs(y2 - y) > ey)[hit].any() and not (np.abs(y2 - y) > ey)[~hit].any()


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers are only safe where no GPU can be reached")
def test_refusals_by_code():
    lib, P = b._lib, ctypes.c_void_p
    A, B, C, odd, n0 = P(1 << 20), P(1 << 22), P(1 << 23), P((1 << 20) + 8), P(None)
    ws, wsn = P(1 << 21), 1 << 26
    DEV = (4, 6)

    def fwd(X=A, ldx=512, ad=A, dn=A, up=A, sc=A, base=C, ldb=264, Y=B, ldy=264, V=n0, M=40, N=264, K=512, r=8, L=2,
            w=ws, n=wsn):
        return lib.cr_lora_forward(X, ldx, ad, dn, up, sc, base, ldb, Y, ldy, V, M, N, K, r, L, w, n, None)

    assert fwd() in DEV and fwd(ad=n0, base=n0, ldb=0) in DEV and fwd(V=A) in DEV
    assert fwd(X=n0, dn=n0, up=n0, sc=n0, Y=n0, base=n0, M=0) in DEV
    assert fwd(X=n0) == 1 and fwd(dn=n0) == 1 and fwd(up=n0) == 1 and fwd(sc=n0) == 1 and fwd(Y=n0) == 1
    assert fwd(base=B) in DEV and fwd(base=B, ldb=272) == 1 and fwd(Y=A) == 1  # in place: the base, with its stride
    assert fwd(M=-1) == 1 and fwd(L=-1) == 1 and fwd(r=-4) == 1 and fwd(ldx=-8) == 1
    assert fwd(r=6) == 2 and fwd(r=0) == 2 and fwd(r=132) == 2 and fwd(L=0) == 2 and fwd(L=4097) == 2
    assert fwd(K=516) == 2 and fwd(N=260) == 2 and fwd(N=0) == 2 and fwd(K=65544, ldx=65544) == 2
    assert fwd(ldx=504) == 1 and fwd(ldy=256) == 1 and fwd(ldb=256) == 1 and fwd(ldb=0) == 1
    assert fwd(ldx=516) == 3 and fwd(X=odd) == 3 and fwd(Y=odd) == 3 and fwd(dn=odd) == 3 and fwd(up=odd) == 3
    assert fwd(base=odd) == 3 and fwd(V=P((1 << 20) + 4)) == 3 and fwd(ad=P((1 << 20) + 2)) == 3
    assert lib.cr_lora_forward_workspace_size(40, 264, 512, 8, 2) == 0 and fwd(w=n0, n=0) in DEV  # few rows: none
    need = lib.cr_lora_forward_workspace_size(4000, 264, 512, 8, 2)
    assert fwd(M=4000, n=need) in DEV and fwd(M=4000, n=need - 1) == 5 and fwd(M=4000, w=n0) == 5
    assert fwd(M=4000, w=P((1 << 21) + 128)) == 5

    def bwd(dY=A, X=A, ldx=512, c=n0, cs=n0, V=A, ad=A, dn=A, up=A, sc=A, base=C, ldb=512, dX=B, lddx=512, dd=A, du=A,
            M=40, N=264, K=512, r=8, L=2, w=ws, n=wsn):
        return lib.cr_lora_backward(dY, 264, X, ldx, c, cs, V, ad, dn, up, sc, base, ldb, dX, lddx, dd, du, M, N, K, r, L,
                                    w, n, None)

    assert bwd() in DEV and bwd(X=n0, ldx=0, c=A, cs=A) in DEV and bwd(X=n0, dd=n0) in DEV and bwd(V=n0, du=n0) in DEV
    assert bwd(dX=n0, dd=n0, du=n0) in DEV
    assert bwd(base=B) in DEV and bwd(base=B, ldb=520) == 1 and bwd(dX=A) == 1 and bwd(dY=B, dX=B) == 1
    assert bwd(c=A, cs=A) == 1  # both X and its checkpoint
    assert bwd(X=n0, c=A) == 1 and bwd(X=n0, cs=A) == 1 and bwd(X=n0) == 1 and bwd(V=n0) == 1 and bwd(sc=n0) == 1
    assert bwd(X=n0, c=A, cs=A, K=520, ldb=520, lddx=520) == 2  # a checkpoint has whole slices
    assert bwd(K=520, ldx=520, ldb=520, lddx=520) in DEV
    assert bwd(dd=odd) == 3 and bwd(du=odd) == 3 and bwd(X=n0, c=odd, cs=A) == 3 and bwd(lddx=508) == 1
    need = lib.cr_lora_backward_workspace_size(40, 264, 512, 8, 2)
    assert bwd(n=need) in DEV and bwd(n=need - 1) == 5

    assert lib.cr_ckpt_save(A, 4, 512, 512, A, A, None) in DEV and lib.cr_ckpt_save(None, 0, 512, 512, None, None, None) in DEV
    assert lib.cr_ckpt_save(None, 4, 512, 512, A, A, None) == 1 and lib.cr_ckpt_save(A, 4, 512, 504, A, A, None) == 1
    assert lib.cr_ckpt_save(A, 4, 520, 520, A, A, None) == 2 and lib.cr_ckpt_save(odd, 4, 512, 512, A, A, None) == 3
    assert lib.cr_ckpt_load(A, A, 4, 512, A, 512, None) in DEV and lib.cr_ckpt_load(A, None, 4, 512, A, 512, None) == 1
    assert lib.cr_ckpt_load(A, A, 4, 128, A, 512, None) == 2 and lib.cr_ckpt_load(A, A, 4, 512, A, 516, None) == 3

    def gi(dY=A, lddy=264, Wq=A, s=A, dX=B, lddx=512, M=40, N=264, K=512, group=256, w=ws, n=wsn):
        return lib.cr_w4a4_grad_input(dY, lddy, Wq, s, dX, lddx, M, N, K, group, w, n, None)

    assert gi() in DEV and gi(M=0, dY=n0, dX=n0) in DEV and gi(N=0, dY=n0, Wq=n0, s=n0) in DEV
    assert gi(dX=A) == 1 and gi(dY=n0) == 1 and gi(Wq=n0) == 1 and gi(s=n0) == 1 and gi(dX=n0) == 1 and gi(lddx=504) == 1
    assert gi(group=32) == 2 and gi(group=1024) == 2 and gi(N=260) == 2 and gi(K=384) == 2
    assert gi(lddy=268) == 3 and gi(dX=odd) == 3
    need = lib.cr_w4a4_grad_input_workspace_size(40, 264, 512, 256)
    assert need >= 40 * 512 * 4 and gi(n=need) in DEV and gi(n=need - 1) == 5
    need = lib.cr_w4a4_grad_input_workspace_size(4, 2640, 512, 256)  # straight from the packed weights
    assert 4 * 2640 * 2 <= need < 2640 * 512 * 2 and gi(M=4, N=2640, lddy=2640, n=need) in DEV
    assert gi(M=4, N=2640, lddy=2640, n=need - 1) == 5
    need = lib.cr_w4a4_grad_input_workspace_size(4000, 264, 512, 256)
    assert need >= 264 * 512 * 2 and gi(M=4000, n=need) in DEV and gi(M=4000, n=need - 1) == 5


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers are only safe where no GPU can be reached")
@pytest.mark.parametrize("M", [0, 40, 4000])
def test_a_given_workspace_is_aligned_whether_the_form_needs_one_or_not(M):
    """The form for few rows needs none, but it writes the status word of one that it is given."""
    lib, P = b._lib, ctypes.c_void_p
    A, B, C = P(1 << 20), P(1 << 22), P(1 << 23)

    def fwd(w, n):
        return lib.cr_lora_forward(A, 512, A, A, A, A, C, 264, B, 264, None, M, 264, 512, 8, 2, w, n, None)

    for off in (1, 2, 4, 8, 16, 128, 255):
        assert fwd(P((1 << 21) + off), 1 << 26) == 5
    assert fwd(P(1 << 21), 1 << 26) in (4, 6)
    assert fwd(None, 0) == (5 if M == 4000 else fwd(P(1 << 21), 1 << 26))


def test_binding_wants_cuda_bf16():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    f = torch.zeros(1, 4, 256, dtype=torch.bfloat16)
    s = torch.ones(1)
    with pytest.raises(TypeError):
        b.cr_lora_forward(x, f, f, s)
    with pytest.raises(TypeError):
        b.cr_lora_backward(x, x, x, f, f, s)
    with pytest.raises(TypeError):
        b.cr_ckpt_save(x)
    with pytest.raises(TypeError):
        b.cr_ckpt_load(torch.zeros(4, 256, dtype=torch.int8), torch.ones(4, 1))
    with pytest.raises(TypeError):
        b.cr_ckpt_load(torch.zeros(4, 256), torch.ones(4, 1))
    with pytest.raises(TypeError):
        b.cr_w4a4_grad_input(x, torch.zeros(256, 128, dtype=torch.uint8), torch.ones(256))


def test_the_other_calls_work_without_the_extension_module():
    """Without _calls the package imports and every ctypes call works; a call that needs it says what is missing."""
    import subprocess
    import sys

    code = """
import sys
sys.modules["w4a8_rotated_quantized_b200._calls"] = None  # what a missing or unloadable module comes to
import torch
import w4a8_rotated_quantized_b200 as cr
assert cr.cr_api_version() == 1 and cr.cr_status_string(0)
x = torch.zeros(4, 256, dtype=torch.bfloat16)
try:
    cr.cr_pack_weight(x.float())
    raise SystemExit("no TypeError")
except TypeError:
    pass
for call in (lambda: cr.cr_ckpt_save(x), lambda: cr.cr_lora_forward(x, x, x, x), lambda: cr.cr_w4a4_grad_input(x, x, x)):
    try:
        call()
        raise SystemExit("no ImportError")
    except ImportError as e:
        assert "_calls" in str(e) and "build" in str(e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_extension_module_is_rebuilt_for_another_torch(monkeypatch):
    from w4a8_rotated_quantized_b200 import build

    assert not build._calls_stale()  # built when the tests were collected
    made = build._calls_made_with()
    assert torch.__version__.split("+")[0] in made
    monkeypatch.setattr(build, "_calls_made_with", lambda: made.replace(torch.__version__.split("+")[0], "0.0"))
    assert build._calls_stale()


def test_timeouts_need_a_place_for_the_answer():
    assert b._lib.cr_read_timeouts(None, None) == 1
    if not torch.cuda.is_available():
        st = ctypes.c_int(-1)
        assert b._lib.cr_read_timeouts(ctypes.byref(st), None) in (4, 6) and st.value == -1
        assert b._lib.cr_selftest_lost_wait(None) in (4, 6)


def test_backward_splits_up_to_the_most_rows():
    """The number of token tiles does not leave 32 bits for the last values of M."""
    size = b._lib.cr_lora_backward_workspace_size
    for N, K, r, L in ((8, 8, 4, 1), (264, 512, 8, 2)):
        most = size(2 ** 31 - 1, N, K, r, L)
        assert most >= size(2 ** 31 - 64, N, K, r, L) > 2 ** 31 * r * 4
        # the partial sums of 2^25 tiles, 512 to a part
        assert most >= 2 ** 31 * r * 4 - 4 * r + 2 ** 16 * L * r * (K + N) * 4
