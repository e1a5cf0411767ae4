"""GPU checks of gdn_gated_rms_norm and gdn_residual_rms_norm against the
formulas in 64 bits.

Bound: half a bf16 step of the result (2^-8 relative) for the final rounding;
the fp32 arithmetic before it is off by at most (n + 40) 2^-24 relative, n the
row's length (its sum of squares, then some ten operations and sigmoids at a
few steps each), of the terms that are added."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import serving_ref as ref

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


def bf(a):
    return torch.tensor(np.asarray(a, np.float32), device="cuda").to(torch.bfloat16)


def near(got, want, terms, n, name):
    err = np.abs(ref.values(got) - want)
    bound = np.abs(want) * HALF + terms * (n + 40) * 2.0 ** -24 * (1 + HALF) + 1e-38
    assert np.isfinite(ref.values(got)).all() and (err <= bound).all(), "%s: %.3g over" % (name, (err - bound).max())


def head_ref(x, w, z, eps, off):
    y = x * ref.rms(x, eps) * (off + w)
    return y if z is None else y * z * ref.sigmoid(z)


@pytest.mark.parametrize("T,H,d", [(1, 1, 8), (3, 2, 16), (5, 6, 40), (7, 3, 64), (1, 32, 128), (33, 4, 136), (20, 16, 256), (9, 1, 504),
                                   (2, 5, 512), (300, 32, 128)])
@pytest.mark.parametrize("gate", [True, False])
def test_head_norm(T, H, d, gate):
    r = np.random.default_rng(T + H + d)
    x, w = bf(r.standard_normal((T, H, d)) * np.exp(2 * r.standard_normal((T, H, 1)))), bf(0.3 * r.standard_normal(d))
    z = bf(3 * r.standard_normal((T, H, d))) if gate else None
    y = torch.full_like(x, 99.0)
    gdn.gdn_gated_rms_norm(x, w, y, gate=z, eps=1e-6, weight_offset=1.0)
    want = head_ref(ref.values(x), ref.values(w), None if z is None else ref.values(z), 1e-6, 1.0)
    near(y, want, np.abs(want), d, "y")


def test_head_norm_views_in_place_and_neighbours():
    r = np.random.default_rng(1)
    wide = bf(r.standard_normal((11, 9, 64)))
    before = wide.clone()
    w = bf(1 + 0.1 * r.standard_normal(64))
    x, z = wide[:, 2:5], wide[:, 6:9]
    want = head_ref(ref.values(x), ref.values(w), ref.values(z), 1e-5, 0.0)
    gdn.gdn_gated_rms_norm(x, w, x, gate=z, eps=1e-5)
    near(x, want, np.abs(want), 64, "y")
    for part in (slice(0, 2), slice(5, 9)):
        assert torch.equal(wide[:, part], before[:, part])


def test_head_norm_extremes():
    """Zero rows give zeros; large values do not overflow before the mean; far gates saturate."""
    x = torch.zeros(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    x[1] = 1e18
    x[2, 0, 7] = -3e18
    x[3] = 1e-20
    z = torch.full((4, 1, 64), 200.0, device="cuda", dtype=torch.bfloat16)
    z[:, :, ::2] = -200.0
    w, y = bf(np.ones(64)), torch.empty_like(x)
    gdn.gdn_gated_rms_norm(x, w, y, gate=z)
    xr, zr = ref.values(x), ref.values(z)
    with np.errstate(over="ignore"):
        want = head_ref(xr, 1.0, zr, 1e-6, 0.0)
    near(y, want, np.abs(want), 64, "y")
    assert (y[0] == 0).all()


def test_head_norm_keeps_bad_rows_apart():
    x = torch.ones(5, 2, 128, device="cuda", dtype=torch.bfloat16)
    x[2, 1, 9] = float("nan")
    x[3, 0, 1] = float("inf")
    y = torch.empty_like(x)
    gdn.gdn_gated_rms_norm(x, bf(np.ones(128)), y)
    bad = ~torch.isfinite(y).all(-1)
    assert bad.nonzero().tolist() == [[2, 1], [3, 0]]


def residual_ref(x, res, pw, z, w, a, eps, off):
    u = x if pw is None else x * ref.rms(x, eps) * (off + pw)
    if z is not None:
        u = u * ref.sigmoid(z)
    h = res + a * u
    return h, h * ref.rms(h, eps) * (off + w), np.abs(res) + np.abs(a * u)


@pytest.mark.parametrize("R,D", [(1, 8), (2, 64), (5, 512), (3, 520), (32, 2048), (4, 2056), (33, 2560), (9, 4096), (3, 4104), (2, 8192),
                                 (3, 8200), (2, 16384), (700, 1024)])
@pytest.mark.parametrize("post,gate", [(False, False), (True, False), (False, True), (True, True)])
def test_residual_norm(R, D, post, gate):
    r = np.random.default_rng(R + D)
    x, res = bf(r.standard_normal((R, D)) * np.exp(r.standard_normal((R, 1)))), bf(2 * r.standard_normal((R, D)))
    w, pw = bf(0.2 * r.standard_normal(D)), bf(0.2 * r.standard_normal(D)) if post else None
    z = bf(2 * r.standard_normal((R, D))) if gate else None
    n, y = torch.full_like(x, 99.0), torch.full_like(x, 99.0)
    gdn.gdn_residual_rms_norm(x, res, w, n, y, post_weight=pw, gate=z, residual_scale=-0.6, eps=1e-5, weight_offset=1.0)
    v = lambda t: None if t is None else ref.values(t)                                  # noqa: E731
    h, want, terms = residual_ref(v(x), v(res), v(pw), v(z), v(w), -0.6, 1e-5, 1.0)
    near(n, h, terms, D, "new_residual")
    near(y, want, terms * ref.rms(h, 1e-5) * np.abs(1.0 + v(w)) + np.abs(want), D, "y")


@pytest.mark.parametrize("place", ["residual", "x", "y_is_x", "both"])
def test_residual_norm_in_place(place):
    r = np.random.default_rng(3)
    x, res, w = bf(r.standard_normal((6, 640))), bf(r.standard_normal((6, 640))), bf(1 + 0.1 * r.standard_normal(640))
    n0, y0 = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_residual_rms_norm(x, res, w, n0, y0, residual_scale=0.5)
    n = {"residual": res, "x": x, "both": res}.get(place, torch.empty_like(x))
    y = x if place in ("y_is_x", "both") else torch.empty_like(x)
    gdn.gdn_residual_rms_norm(x, res, w, n, y, residual_scale=0.5)
    assert torch.equal(n, n0) and torch.equal(y, y0)


def test_residual_norm_strided_rows_and_neighbours():
    r = np.random.default_rng(4)
    wide = bf(r.standard_normal((7, 4 * 264)))
    before = wide.clone()
    col = lambda i: wide[:, 264 * i: 264 * i + 256]                                      # noqa: E731
    x, res, n, y = (col(i) for i in range(4))
    w = bf(np.ones(256))
    h, want, terms = residual_ref(ref.values(x), ref.values(res), None, None, np.ones(256), 1.0, 1e-6, 0.0)
    gdn.gdn_residual_rms_norm(x, res, w, n, y)
    near(n, h, terms, 256, "new_residual")
    near(y, want, terms * ref.rms(h, 1e-6) + np.abs(want), 256, "y")
    for i in range(4):
        assert torch.equal(wide[:, 264 * i + 256: 264 * (i + 1)], before[:, 264 * i + 256: 264 * (i + 1)])
    assert torch.equal(x, before[:, :256])


def test_residual_norm_zero_rows():
    x = torch.zeros(3, 128, device="cuda", dtype=torch.bfloat16)
    n, y = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_residual_rms_norm(x, x.clone(), bf(np.ones(128)), n, y, post_weight=bf(np.ones(128)))
    assert (n == 0).all() and (y == 0).all()


def test_in_a_graph():
    r = np.random.default_rng(5)
    x, res, w, z = bf(r.standard_normal((33, 2560))), bf(r.standard_normal((33, 2560))), bf(np.ones(2560)), bf(r.standard_normal((33, 2560)))
    n, y, hy = torch.empty_like(x), torch.empty_like(x), torch.empty(33, 20, 128, dtype=torch.bfloat16, device="cuda")

    def step():
        gdn.gdn_residual_rms_norm(x, res, w, n, y, post_weight=w, gate=z)
        gdn.gdn_gated_rms_norm(y.view(33, 20, 128), w[:128], hy, gate=z.view(33, 20, 128))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        x.copy_(bf(r.standard_normal((33, 2560))))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (n, y, hy)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (n, y, hy)))
