"""Layer norm (forward, backward) and the mixture-of-experts decode step.

CPU: the oracle's formulas against float64 autograd and brute force, and the
library's refusals.  GPU: every output element within a bound counted from
its arithmetic: half a rounding step of the output type (relative 2^-8 for
bf16, 2^-24 for fp32) plus 2^-24 (2^-23 for a matrix instruction's
accumulation) times the number of additions on the longest path times the sum
of the terms' magnitudes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import associative_algebra_block_b200 as aal
from associative_algebra_block_b200 import inputs

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
FAKE = 0x10000  # never dereferenced: the calls below fail validation first


# ------------------------------------------------------------------ the oracle
def test_layer_norm_oracle_equals_float64_autograd():
    rng = np.random.default_rng(3)
    S, dY = rng.normal(1.0, 2.0, (5, 7)), rng.normal(size=(5, 7))
    gamma, beta = rng.normal(size=7), rng.normal(size=7)
    St, gt, bt = (torch.tensor(v, requires_grad=True) for v in (S, gamma, beta))
    Y = torch.nn.functional.layer_norm(St, (7,), gt, bt, 1e-5)
    Y.backward(torch.tensor(dY))
    got, mean, rstd = oracle.layer_norm(S, gamma, beta, 1e-5)
    assert np.allclose(got, Y.detach().numpy(), rtol=0, atol=1e-12)
    for g, t in zip(oracle.layer_norm_bwd(S, gamma, mean, rstd, dY), (St, gt, bt)):
        assert np.allclose(g, t.grad.numpy(), rtol=0, atol=1e-12)


def test_layer_norm_oracle_gradient_equals_differences():
    rng = np.random.default_rng(4)
    S, dY, gamma = rng.normal(size=(2, 6)), rng.normal(size=(2, 6)), rng.normal(size=6)
    _, mean, rstd = oracle.layer_norm(S, gamma)
    dS, _, _ = oracle.layer_norm_bwd(S, gamma, mean, rstd, dY)
    for i in range(2):
        for j in range(6):
            up, dn = S.copy(), S.copy()
            up[i, j] += 1e-6
            dn[i, j] -= 1e-6
            diff = ((oracle.layer_norm(up, gamma)[0] - oracle.layer_norm(dn, gamma)[0]) * dY).sum() / 2e-6
            assert abs(diff - dS[i, j]) <= 1e-7


def test_moe_oracle_equals_brute_force_and_breaks_ties_low():
    rng = np.random.default_rng(5)
    B, D, F, E, k = 3, 4, 6, 5, 2
    x, Wr = rng.normal(size=(B, D)), rng.normal(size=(D, E))
    Wr[:, 4] = Wr[:, 1]  # experts 1 and 4 tie everywhere
    Wg, Wu, Wd = rng.normal(size=(E * D, F)), rng.normal(size=(E * D, F)), rng.normal(size=(E * F, D))
    Y, ids, w = oracle.moe_decode("Q", 1, np.zeros(B, np.int64), x, Wr, Wg, Wu, Wd, k)
    for b in range(B):
        logits = [float(x[b] @ Wr[:, e]) for e in range(E)]
        want = sorted(range(E), key=lambda e: (-logits[e], e))[:k]
        assert list(ids[b]) == want and not (4 in want and 1 not in want)
        p = np.exp([logits[e] for e in want])
        out = np.zeros(D)
        for e, pe in zip(want, p / p.sum()):
            g, u = x[b] @ Wg[e * D:(e + 1) * D], x[b] @ Wu[e * D:(e + 1) * D]
            out += pe * ((g / (1 + np.exp(-g)) * u) @ Wd[e * F:(e + 1) * F])
        assert np.allclose(Y[b], out, rtol=0, atol=1e-12)
    _, w_all = oracle.route(x, Wr, k, renormalize=False)
    assert (w_all.sum(1) < 1).all() and np.allclose(w_all / w_all.sum(1, keepdims=True), w)


# ------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(aal.LIB_PATH):
        from associative_algebra_block_b200 import build
        build.build()
    return aal.load()


def _m(ptr, rows, cols, ld=None, dtype=aal.AAL_BF16):
    return aal.AalMat(ptr, dtype, rows, cols, cols if ld is None else ld)


NONE = aal.AalMat(None, aal.AAL_BF16, 0, 0, 0)
BAD, UNS = aal.AAL_ERR_INVALID_ARG, aal.AAL_ERR_UNSUPPORTED


def test_layer_norm_refusals(lib):
    X, Y, g = _m(FAKE, 4, 8), _m(FAKE + 4096, 4, 8), _m(FAKE, 1, 8)
    f32 = aal.AAL_F32

    def fwd(X=X, R=NONE, g=g, b=g, eps=1e-5, S=NONE, Y=Y, mean=None, rstd=None):
        return lib.aal_layer_norm_fwd(X, R, g, b, eps, S, Y, mean, rstd, None)

    assert fwd(Y=_m(FAKE, 4, 9)) == BAD
    assert fwd(X=_m(None, 4, 8)) == BAD
    assert fwd(R=_m(FAKE, 3, 8)) == BAD
    assert fwd(S=_m(FAKE, 4, 8)) == BAD                           # S without R
    assert fwd(R=X, S=_m(FAKE + 4096, 4, 8)) == BAD               # S is Y
    assert fwd(g=_m(FAKE, 1, 7)) == BAD and fwd(b=_m(FAKE, 2, 8)) == BAD
    assert fwd(eps=-1.0) == BAD and fwd(eps=float("nan")) == BAD and fwd(eps=float("inf")) == BAD
    assert fwd(mean=FAKE + 2) == BAD and fwd(rstd=FAKE + 1) == BAD
    assert fwd(Y=_m(FAKE, 4, 8, dtype=f32)) == UNS
    assert fwd(g=_m(FAKE, 1, 8, dtype=f32)) == UNS                # gamma fp32, beta bf16
    assert fwd(X=_m(FAKE, 4, 8, dtype=f32), Y=_m(FAKE, 4, 8, dtype=f32)) == BAD  # bf16 parameters, fp32 rows
    assert fwd(X=_m(None, 0, 8), Y=_m(None, 0, 8)) == aal.AAL_OK

    def bwd(X=X, g=g, mean=FAKE, rstd=FAKE, dY=Y, dR=NONE, dX=X, dg=g, db=_m(FAKE + 64, 1, 8)):
        return lib.aal_layer_norm_bwd(X, g, mean, rstd, dY, dR, dX, dg, db, 0, None)

    assert bwd(dY=_m(FAKE, 4, 9)) == BAD and bwd(dX=_m(FAKE, 5, 8)) == BAD
    assert bwd(mean=None) == BAD and bwd(rstd=None) == BAD and bwd(mean=FAKE + 2) == BAD
    assert bwd(dR=Y, dX=NONE) == BAD                               # a residual gradient with nowhere to go
    assert bwd(dg=_m(FAKE, 1, 9)) == BAD and bwd(dg=_m(FAKE, 1, 8, dtype=f32)) == BAD
    assert bwd(dg=g, db=g) == BAD                                  # both gradients in one place
    assert bwd(dY=_m(FAKE, 4, 8, dtype=f32)) == UNS
    assert bwd(dX=NONE, dg=NONE, db=NONE) == aal.AAL_OK            # nothing asked for
    assert lib.aal_layer_norm_bwd_workspace_size(-1, 8) == -1
    assert aal.aal_layer_norm_bwd_workspace_size(0, 8) == 0
    assert aal.aal_layer_norm_bwd_workspace_size(1, 64) >= 64 * 2 * 4
    with pytest.raises(ValueError):
        aal.aal_layer_norm_bwd_workspace_size(4, -1)


def test_moe_refusals(lib):
    B, D, F, E, k = 2, 8, 12, 4, 2
    good = dict(law=0, q=2, pos=FAKE, x=_m(FAKE, B, D), wr=_m(FAKE, D, E), wg=_m(FAKE, E * D, F), wu=_m(FAKE, E * D, F),
                wd=_m(FAKE, E * F, D), r=NONE, k=k, ids=FAKE, w=FAKE, h=_m(FAKE, B * k, F), y=_m(FAKE, B, D))

    def call(**kw):
        a = dict(good, **kw)
        return lib.aal_moe_decode(a["law"], a["q"], a["pos"], a["x"], a["wr"], a["wg"], a["wu"], a["wd"], a["r"], a["k"],
                                  1, a["ids"], a["w"], a["h"], a["y"], None)

    f32 = aal.AAL_F32
    for bad in (dict(law=1), dict(q=0), dict(q=3), dict(pos=None), dict(pos=FAKE + 4), dict(ids=None), dict(w=None),
                dict(ids=FAKE + 2), dict(w=FAKE + 2), dict(k=0), dict(k=E + 1), dict(wr=_m(FAKE, D + 1, E)),
                dict(wg=_m(FAKE, E * D - 1, F)), dict(wu=_m(FAKE, E * D, F + 2)), dict(wd=_m(FAKE, E * F, D - 2)),
                dict(r=_m(FAKE, B, D + 1)), dict(h=_m(FAKE, B, F)), dict(y=_m(FAKE, B + 1, D)), dict(x=_m(None, B, D)),
                dict(wr=_m(FAKE, D, 0))):
        assert call(**bad) == BAD, bad
    for bad in (dict(wr=_m(FAKE, D, E, dtype=f32)), dict(r=_m(FAKE, B, D, dtype=f32)), dict(h=_m(FAKE, B * k, F, dtype=f32))):
        assert call(**bad) == UNS, bad
    # more experts or choices than the router holds
    assert call(wr=_m(FAKE, D, 2049), wg=_m(FAKE, 2049 * D, F), wu=_m(FAKE, 2049 * D, F), wd=_m(FAKE, 2049 * F, D)) == UNS
    assert call(wr=_m(FAKE, D, 64), wg=_m(FAKE, 64 * D, F), wu=_m(FAKE, 64 * D, F), wd=_m(FAKE, 64 * F, D), k=33,
                h=_m(FAKE, B * 33, F)) == UNS
    wide = 2 ** 20 + 2
    assert call(wg=_m(FAKE, E * D, wide), wu=_m(FAKE, E * D, wide), wd=_m(FAKE, E * wide, D), h=_m(FAKE, B * k, wide)) == UNS
    # nothing to do: no entries
    assert call(pos=None, x=_m(None, 0, D), ids=None, w=None, h=_m(None, 0, F), y=_m(None, 0, D)) == aal.AAL_OK


def test_bindings_refuse_wrong_tensors(lib):
    z = torch.empty(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        aal.aal_layer_norm_fwd(z, None, None, z)
    e = torch.empty(0, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="1-D"):
        aal.aal_layer_norm_fwd(e, torch.empty(0, 8), None, e)
    with pytest.raises(ValueError, match="float32"):
        aal.aal_layer_norm_fwd(e, None, None, e, mean=torch.empty(0, dtype=torch.float64))
    with pytest.raises(ValueError, match="no entries"):  # empty is not left out
        aal.aal_layer_norm_bwd(e, torch.empty(0), torch.empty(0), torch.empty(0), e)
    with pytest.raises(ValueError, match="entries"):
        aal.aal_layer_norm_bwd(e, None, torch.empty(3), torch.empty(0), e)
    pos = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA device"):
        aal.aal_moe_decode("Q", 1, pos, z, z, z, z, z, torch.empty(4, 2, dtype=torch.int32), torch.empty(4, 2), z, z)
    pos, w0 = torch.empty(0, dtype=torch.int64), torch.empty(0, 0, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ids"):
        aal.aal_moe_decode("Q", 1, pos, e, w0, w0, w0, w0, torch.empty(3, 2, dtype=torch.int32), torch.empty(0, 2), e, e)
    # empty tensors reach the library without a GPU and launch nothing
    aal.aal_launch_count(reset=True)
    aal.aal_layer_norm_fwd(e, None, None, e)
    aal.aal_layer_norm_bwd(e, None, torch.empty(0), torch.empty(0), e)
    assert aal.aal_launch_count() == 0


# -------------------------------------------------------------- GPU, layer norm
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    aal.load()


def h64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _strided(m, d, dtype, ld, fill=None, seed=0, scale=1.0, shift=0.0):
    """[m, d] view of a wider buffer, and the buffer: what lies outside the
    view must stay as it was."""
    big = torch.full((m, ld), 7.25, dtype=TD[dtype], device="cuda")
    v = big[:, :d]
    if fill is None:
        gen = torch.Generator().manual_seed(seed)
        v.copy_(torch.randn(m, d, generator=gen) * scale + shift)
    else:
        v.fill_(fill)
    return v, big


def _outside_kept(big, d):
    return bool((big[:, d:] == 7.25).all())


# sizes around one vector, one warp row, the block path, odd widths (element
# by element), several rows a CTA, and a row wider than the registers hold
LN_SIZES = [(1, 1), (1, 768), (3, 8), (5, 17), (9, 64), (33, 257), (70, 768), (19, 1000), (600, 1003), (4, 1024),
            (37, 1032), (6, 4096), (3, 8200), (2, 16384), (2, 33000), (2, 20001), (5000, 40)]


def _bound_terms(d):
    return (d / 32 + 64) * 2.0 ** -24  # additions on the longest path: a thread's own and two trees


@gpu
@pytest.mark.parametrize("dtype,affine", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", None)])
@pytest.mark.parametrize("m,d", LN_SIZES)
def test_layer_norm_fwd(cuda, m, d, dtype, affine):
    res = (m + d) % 2 == 0
    ld = d + (8 if d % 8 == 0 and d % 3 else 0) + (1 if d % 5 == 2 else 0)
    X, _ = _strided(m, d, dtype, ld, seed=m + d, scale=3.0, shift=5.0)
    R, _ = _strided(m, d, dtype, ld, seed=m + d + 1) if res else (None, None)
    Y, Yb = _strided(m, d, dtype, ld, fill=float("nan"))
    S, Sb = _strided(m, d, dtype, ld, fill=float("nan")) if res else (None, None)
    gen = torch.Generator().manual_seed(9)
    gamma = beta = None
    if affine:
        gamma = (torch.randn(d, generator=gen) + 1).to(TD[affine]).cuda()
        beta = torch.randn(d, generator=gen).to(TD[affine]).cuda()
    mean, rstd = (torch.full((m,), float("nan"), device="cuda") for _ in range(2))
    aal.aal_layer_norm_fwd(X, gamma, beta, Y, 1e-5, R=R, S=S, mean=mean, rstd=rstd)
    s = h64(X) + (h64(R) if res else 0.0)
    g64, b64 = (h64(gamma), h64(beta)) if affine else (None, None)
    ref, mu, rs = oracle.layer_norm(s, g64, b64, 1e-5)
    e = _bound_terms(d)
    big = np.abs(s).max(1)
    assert (np.abs(h64(mean) - mu) <= e * big).all()
    # var's relative error: 2 e (the squares) + the mean's error against the spread, squared or crossed
    var = ((s - mu[:, None]) ** 2).mean(1) + 1e-5
    rel = 2 * e + 2 * e * big / np.sqrt(var) + (e * big) ** 2 / var + 4 * 2.0 ** -24
    assert (np.abs(h64(rstd) - rs) <= rel * rs).all()
    ga = np.abs(g64) if affine else 1.0
    err = (e * big * rs)[:, None] * ga + (rel + 8 * 2.0 ** -24)[:, None] * np.abs((s - mu[:, None]) * rs[:, None]) * ga
    err = err + 2.0 ** -23 * np.abs(ref) + 2.0 ** -23 * (np.abs(b64) if affine else 0.0)
    assert (np.abs(h64(Y) - ref) <= HALF[dtype] * np.abs(ref) + 1.01 * err).all()
    assert _outside_kept(Yb, d)
    if res:
        assert (np.abs(h64(S) - s) <= HALF[dtype] * np.abs(s) * 1.01).all() and _outside_kept(Sb, d)


@gpu
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("dtype,affine", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", None)])
@pytest.mark.parametrize("m,d", LN_SIZES)
def test_layer_norm_bwd(cuda, m, d, dtype, affine, ws):
    res = (m + d) % 2 == 1
    ld = d + (16 if d % 8 == 0 and d % 3 else 0) + (3 if d % 5 == 2 else 0)
    X, _ = _strided(m, d, dtype, ld, seed=m + d, scale=2.0, shift=1.0)
    dY, _ = _strided(m, d, dtype, ld, seed=m + d + 1)
    dR, _ = _strided(m, d, dtype, ld, seed=m + d + 2) if res else (None, None)
    dX, dXb = _strided(m, d, dtype, ld, fill=float("nan"))
    gen = torch.Generator().manual_seed(9)
    pt = TD[affine] if affine else TD[dtype]
    gamma = (torch.randn(d, generator=gen) + 1).to(pt).cuda() if affine else None
    _, mu, rs = oracle.layer_norm(h64(X))
    mean, rstd = (torch.from_numpy(v).float().cuda() for v in (mu, rs))
    dgamma, dbeta = (torch.full((d,), float("nan"), dtype=pt, device="cuda") for _ in range(2))
    buf = torch.empty(max(1, aal.aal_layer_norm_bwd_workspace_size(m, d)), dtype=torch.uint8, device="cuda")
    aal.aal_set_workspace(buf if ws else None)
    try:
        aal.aal_layer_norm_bwd(X, gamma, mean, rstd, dY, dX=dX, dgamma=dgamma, dbeta=dbeta, dR=dR)
    finally:
        aal.aal_set_workspace(None)
    mu, rs = h64(mean), h64(rstd)
    g64 = h64(gamma) if affine else None
    ref, rg, rb = oracle.layer_norm_bwd(h64(X), g64, mu, rs, h64(dY))
    if res:
        ref = ref + h64(dR)
    xh = (h64(X) - mu[:, None]) * rs[:, None]
    g = h64(dY) * (g64 if affine else 1.0)
    e = _bound_terms(d) + 8 * 2.0 ** -24
    # x - mean rounds against |x|, so xh is off by 2^-23 |x| rstd
    dxh = 2.0 ** -23 * (np.abs(h64(X)) + np.abs(mu)[:, None]) * rs[:, None] + 2.0 ** -23 * np.abs(xh)
    mgx, mg = np.abs(g * xh).mean(1)[:, None], np.abs(g).mean(1)[:, None]
    err = rs[:, None] * (e * (np.abs(g) + mg + np.abs(xh) * mgx) + np.abs(xh) * (np.abs(g) * dxh).mean(1)[:, None] + dxh * mgx)
    err = err + 2.0 ** -23 * np.abs(ref)
    assert (np.abs(h64(dX) - ref) <= HALF[dtype] * np.abs(ref) + 1.01 * err).all()
    assert _outside_kept(dXb, d)
    half = HALF[affine or dtype]
    n = (m / 32 + 64 + min(m, 600)) * 2.0 ** -24  # additions of a column on its longest path, at most
    ag, ab = np.abs(h64(dY) * xh).sum(0), np.abs(h64(dY)).sum(0)
    assert (np.abs(h64(dgamma) - rg) <= half * np.abs(rg) + n * ag + (np.abs(h64(dY)) * dxh).sum(0) + 1e-30).all()
    assert (np.abs(h64(dbeta) - rb) <= half * np.abs(rb) + n * ab + 1e-30).all()


@gpu
def test_layer_norm_bwd_accumulates_and_skips_what_is_not_asked(cuda):
    X, _ = _strided(65, 96, "f32", 96, seed=1)
    dY, _ = _strided(65, 96, "f32", 96, seed=2)
    _, mu, rs = oracle.layer_norm(h64(X))
    mean, rstd = (torch.from_numpy(v).float().cuda() for v in (mu, rs))
    buf = torch.empty(aal.aal_layer_norm_bwd_workspace_size(65, 96), dtype=torch.uint8, device="cuda")
    outs = []
    for ws in (buf, None):
        aal.aal_set_workspace(ws)
        try:
            dg, db = torch.zeros(96, device="cuda"), torch.zeros(96, device="cuda")
            aal.aal_layer_norm_bwd(X, None, mean, rstd, dY, dgamma=dg, dbeta=db)
            dg2, db2 = dg + 1, db - 2
            aal.aal_layer_norm_bwd(X, None, mean, rstd, dY, dgamma=dg2, dbeta=db2, accumulate=True)
            assert torch.allclose(dg2, 2 * dg + 1, atol=1e-4) and torch.allclose(db2, 2 * db - 2, atol=1e-4)
            only = torch.zeros(96, device="cuda")
            aal.aal_layer_norm_bwd(X, None, mean, rstd, dY, dbeta=only)
            assert torch.equal(only, db)
            dx1, dx2 = torch.empty_like(X), dY.clone()
            aal.aal_layer_norm_bwd(X, None, mean, rstd, dY, dX=dx1)
            dg3 = torch.empty_like(dg)
            aal.aal_layer_norm_bwd(X, None, mean, rstd, dx2, dX=dx2, dgamma=dg3)  # dX over dY
            assert torch.equal(dx1, dx2) and torch.equal(dg3, dg)
            # no rows: zero, or unchanged when accumulating
            e = torch.empty(0, 96, device="cuda")
            z = torch.empty(0, device="cuda")
            gz, gk = torch.full((96,), 3.0, device="cuda"), torch.full((96,), 3.0, device="cuda")
            aal.aal_layer_norm_bwd(e, None, z, z, e, dgamma=gz)
            aal.aal_layer_norm_bwd(e, None, z, z, e, dgamma=gk, accumulate=True)
            assert (gz == 0).all() and (gk == 3).all()
        finally:
            aal.aal_set_workspace(None)
        outs.append(dg)
    assert torch.allclose(outs[0], outs[1], atol=1e-4)


@gpu
@pytest.mark.parametrize("d", [768, 1003, 33000])
def test_layer_norm_in_place_and_special_rows(cuda, d):
    X, _ = _strided(6, d, "bf16", d, seed=3)
    R, _ = _strided(6, d, "bf16", d, seed=4)
    X[1], R[1] = 2.5, 0.0            # a constant row: y = beta
    X[2, 3] = float("inf")
    X[3, 0] = float("nan")
    Y, S = torch.empty_like(X), torch.empty_like(X)
    beta = torch.randn(d, device="cuda")
    aal.aal_layer_norm_fwd(X, None, beta, Y, R=R, S=S)
    assert torch.equal(Y[1].float(), beta.bfloat16().float())
    assert torch.isnan(Y[2]).all() and torch.isnan(Y[3]).all()  # the row itself, and only it
    assert torch.isfinite(Y[[0, 1, 4, 5]]).all()
    Xa, Ra = X.clone(), R.clone()
    aal.aal_layer_norm_fwd(Xa, None, beta, Ra, R=Ra, S=Xa)      # the sum over X, the norm over R
    assert torch.equal(Xa.nan_to_num(9), S.nan_to_num(9)) and torch.equal(Ra.nan_to_num(9), Y.nan_to_num(9))
    Xb = X.clone()
    aal.aal_layer_norm_fwd(Xb, None, beta, Xb)
    Yb = torch.empty_like(X)
    aal.aal_layer_norm_fwd(X, None, beta, Yb)
    assert torch.equal(Xb.nan_to_num(9), Yb.nan_to_num(9))


# rows of several widths, many of them, back to back and odd in number: the
# forms in which a warp takes several rows or a copy brings them at once
@gpu
@pytest.mark.parametrize("m,d,dtype", [(4097, 48, "bf16"), (1001, 96, "bf16"), (4099, 32, "f32"), (2051, 200, "bf16"),
                                       (9001, 24, "f32"), (7, 128, "bf16"), (2501, 768, "bf16"), (1203, 2048, "bf16"),
                                       (903, 333, "bf16"), (801, 1501, "f32"), (403, 5001, "bf16"), (300, 7000, "f32")])
def test_layer_norm_many_contiguous_rows(cuda, m, d, dtype):
    gen = torch.Generator().manual_seed(m + d)
    X, R, dY = (torch.randn(m, d, generator=gen).to(TD[dtype]).cuda() for _ in range(3))
    gamma, beta = (torch.randn(d, generator=gen).cuda() for _ in range(2))
    Y, S, dX = (torch.full_like(X, float("nan")) for _ in range(3))
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    aal.aal_layer_norm_fwd(X, gamma, beta, Y, R=R, S=S, mean=mean, rstd=rstd)
    s = h64(X) + h64(R)
    ref, mu, rs = oracle.layer_norm(s, h64(gamma), h64(beta))
    e = 4 * _bound_terms(d)  # the mean, the variance (twice the mean's part) and the product
    scale = np.abs(s).max(1)[:, None] * rs[:, None] * np.abs(h64(gamma)) + np.abs(h64(beta))
    assert (np.abs(h64(Y) - ref) <= HALF[dtype] * np.abs(ref) + e * scale).all()
    assert (np.abs(h64(S) - s) <= HALF[dtype] * np.abs(s) * 1.01).all()
    dg, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    buf = torch.empty(aal.aal_layer_norm_bwd_workspace_size(m, d), dtype=torch.uint8, device="cuda")
    aal.aal_set_workspace(buf)
    try:
        aal.aal_layer_norm_bwd(S, gamma, mean, rstd, dY, dX=dX, dgamma=dg, dbeta=db, dR=R)
        again = torch.empty_like(dg)
        aal.aal_layer_norm_bwd(S, gamma, mean, rstd, dY, dX=dX, dgamma=again, dbeta=db, dR=R)
    finally:
        aal.aal_set_workspace(None)
    assert torch.equal(dg, again)  # the same sums in the same order
    rx, rg, rb = oracle.layer_norm_bwd(h64(S), h64(gamma), h64(mean), h64(rstd), h64(dY))
    xh = np.abs((h64(S) - h64(mean)[:, None]) * h64(rstd)[:, None])
    g = np.abs(h64(dY) * h64(gamma))
    mag = h64(rstd)[:, None] * (g + g.mean(1)[:, None] + (xh + np.abs(h64(mean) * h64(rstd))[:, None]) * (g * xh).mean(1)[:, None])
    assert (np.abs(h64(dX) - rx - h64(R)) <= HALF[dtype] * np.abs(rx + h64(R)) + 4 * _bound_terms(d) * (mag + np.abs(h64(R)))).all()
    n = (m / 32 + 700) * 2.0 ** -24
    assert (np.abs(h64(dg) - rg) <= n * (np.abs(h64(dY)) * (xh + 1)).sum(0)).all()
    assert (np.abs(h64(db) - rb) <= n * np.abs(h64(dY)).sum(0)).all()


# every matrix at an alignment and a stride of its own
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [5, 64, 700, 1500])
def test_layer_norm_mixed_alignments(cuda, d, dtype):
    m = 37

    def at(off, ld, seed):
        big = torch.full((m, ld), 7.25, dtype=TD[dtype], device="cuda")
        v = big[:, off:off + d]
        v.copy_(torch.randn(m, d, generator=torch.Generator().manual_seed(seed)))
        return v, big

    X, _ = at(0, d + 8, 1)
    R, _ = at(3, d + 5, 2)
    S, Sb = at(1, d + 2, 3)
    Y, Yb = at(7, d + 9, 4)
    aal.aal_layer_norm_fwd(X, None, None, Y, R=R, S=S)
    Xc, Rc, Yc, Sc = X.contiguous(), R.contiguous(), torch.empty(m, d, dtype=TD[dtype], device="cuda"), torch.empty(
        m, d, dtype=TD[dtype], device="cuda")
    ref, mu, rs = oracle.layer_norm(h64(Xc) + h64(Rc))
    tol = HALF[dtype] * np.abs(ref) + 8 * _bound_terms(d) * (np.abs(h64(Xc) + h64(Rc)).max(1) * rs)[:, None]
    assert (np.abs(h64(Y) - ref) <= tol).all()
    assert (Yb[:, :7] == 7.25).all() and (Yb[:, 7 + d:] == 7.25).all() and (Sb[:, :1] == 7.25).all() and (Sb[:, 1 + d:] == 7.25).all()
    aal.aal_layer_norm_fwd(Xc, None, None, Yc, R=Rc, S=Sc)
    assert torch.equal(S, Sc)
    dX, dXb = at(5, d + 11, 5)
    mean, rstd = torch.from_numpy(mu).float().cuda(), torch.from_numpy(rs).float().cuda()
    dg = torch.empty(d, device="cuda")
    aal.aal_layer_norm_bwd(S, None, mean, rstd, X, dX=dX, dgamma=dg, dR=R)
    rx, rg, _ = oracle.layer_norm_bwd(h64(S), None, h64(mean), h64(rstd), h64(X))
    assert np.abs(h64(dX) - rx - h64(R)).max() <= HALF[dtype] * np.abs(rx + h64(R)).max() + 64 * _bound_terms(d)
    assert np.abs(h64(dg) - rg).max() <= 200 * 2.0 ** -24 * np.abs(h64(X)).sum(0).max() * 4
    assert (dXb[:, :5] == 7.25).all() and (dXb[:, 5 + d:] == 7.25).all()


@gpu
def test_layer_norm_offsets_past_32_bits(cuda):
    # rows 2^31 elements apart: the second row starts past a 32-bit offset
    ld = 1 << 31
    big = torch.empty(ld + 64, dtype=torch.bfloat16, device="cuda")
    X = torch.as_strided(big, (2, 64), (ld, 1))
    X.copy_(torch.randn(2, 64, generator=torch.Generator().manual_seed(0)))
    Y = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
    aal.aal_layer_norm_fwd(X, None, None, Y)
    ref, _, _ = oracle.layer_norm(h64(X))
    assert (np.abs(h64(Y) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5).all()


@gpu
def test_layer_norm_autograd_and_block(cuda):
    law, q, M, D, F = "Q2xQ2", 4, 256, 64, 128
    s = inputs.Stream(11)
    X = s.normal(M, D, 1.0, "f32").t.cuda().requires_grad_(True)
    Wg, Wu = (s.normal(D, F, D ** -0.5, "f32").t.cuda().requires_grad_(True) for _ in range(2))
    Wd = s.normal(F, D, F ** -0.5, "f32").t.cuda().requires_grad_(True)
    gamma = (1 + 0.1 * torch.randn(D, device="cuda")).requires_grad_(True)
    beta = (0.1 * torch.randn(D, device="cuda")).requires_grad_(True)
    from associative_algebra_block_b200.autograd import layer_norm, swiglu_block
    dY = s.normal(M, D, 1.0, "f32")
    swiglu_block(law, q, aal.row_rule(seq_len=64), X, gamma, beta, Wg, Wu, Wd).backward(dY.t.cuda())
    types = oracle.row_types(law, q, inputs.packed_positions(M, 64))
    N, mean, rstd = oracle.layer_norm(h64(X), h64(gamma), h64(beta))
    dN, dWg, dWu, dWd = oracle.swiglu_bwd(law, q, types, N, h64(Wg), h64(Wu), h64(Wd), dY.f64)
    dS, dg, db = oracle.layer_norm_bwd(h64(X), h64(gamma), mean, rstd, dN)
    for got, ref in ((X.grad, dS + dY.f64), (gamma.grad, dg), (beta.grad, db), (Wg.grad, dWg), (Wd.grad, dWd)):
        assert oracle.rel_err(h64(got), ref) <= 1e-5
    # with a residual: both outputs carry a gradient
    A, B = (s.normal(8, D, 1.0, "f32").t.cuda().requires_grad_(True) for _ in range(2))
    Y, S = layer_norm(A, gamma, beta, residual=B)
    w1, w2 = s.normal(8, D, 1.0, "f32"), s.normal(8, D, 1.0, "f32")
    (Y * w1.t.cuda() + S * w2.t.cuda()).sum().backward()
    s64 = h64(A) + h64(B)
    _, mean, rstd = oracle.layer_norm(s64)
    dS, _, _ = oracle.layer_norm_bwd(s64, h64(gamma), mean, rstd, w1.f64)
    assert oracle.rel_err(h64(A.grad), dS + w2.f64) <= 1e-5 and torch.equal(A.grad, B.grad)


# ------------------------------------------------------------------- GPU, experts
class Moe:
    def __init__(self, B, E, k, D, F, law, q, dtype, seed=0, pad=0, residual=True):
        s = inputs.Stream(seed)
        self.law, self.q, self.B, self.E, self.k, self.D, self.F, self.dtype = law, q, B, E, k, D, F, dtype

        def mk(r, c, sigma):
            t = s.normal(r, c, sigma, dtype, want_f64=False).t
            big = torch.full((r, c + pad), 7.25, dtype=t.dtype, device="cuda")
            big[:, :c] = t.cuda()
            return big[:, :c]

        self.x, self.Wr = mk(B, D, 1.0), mk(D, E, D ** -0.5)
        self.Wg, self.Wu, self.Wd = mk(E * D, F, D ** -0.5), mk(E * D, F, D ** -0.5), mk(E * F, D, F ** -0.5)
        self.R = mk(B, D, 1.0) if residual else None
        self.pos = torch.from_numpy(s.positions(B, 1536)).cuda()
        self.ids = torch.full((B, k), -7, dtype=torch.int32, device="cuda")
        self.w = torch.full((B, k), float("nan"), device="cuda")
        self.h, self.y = mk(B * k, F, 1.0), mk(B, D, 1.0)

    def run(self, **kw):
        aal.aal_moe_decode(self.law, self.q, self.pos, self.x, self.Wr, self.Wg, self.Wu, self.Wd, self.ids, self.w, self.h,
                           self.y, R=self.R, **kw)

    def check(self, renormalize=True, rows=None):
        """Every element against the oracle within the counted bound."""
        law, q, D, F = self.law, self.q, self.D, self.F
        rows = np.arange(self.B) if rows is None else rows
        x, Wr = h64(self.x)[rows], h64(self.Wr)
        pos = self.pos.cpu().numpy()[rows]
        ids, w = oracle.route(x, Wr, self.k, renormalize)
        assert np.array_equal(self.ids.cpu().numpy()[rows], ids)
        assert (np.abs(h64(self.w)[rows] - w) <= 64 * 2.0 ** -24 * w + 1e-38).all()
        half = HALF[self.dtype]
        u23 = 2.0 ** -23
        R = h64(self.R)[rows] if self.R is not None else np.zeros((len(rows), D))
        y, err, mag = R.copy(), np.zeros_like(R), np.abs(R)
        for e in np.unique(ids):
            r, j = np.nonzero(ids == e)
            Wg, Wu = h64(self.Wg[e * D:(e + 1) * D]), h64(self.Wu[e * D:(e + 1) * D])
            Wd = h64(self.Wd[e * F:(e + 1) * F])
            g, u = oracle.decode(law, q, pos[r], x[r], Wg), oracle.decode(law, q, pos[r], x[r], Wu)
            # additions on the longest path: all K of them at most one by one
            # in the general kernel (K / 8 a warp), K / 16 in the matrix path
            n_in, n_out = (D / 8 + 32) * u23, (F / 8 + 32) * u23
            dg = n_in * oracle.decode(law, q, pos[r], np.abs(x[r]), np.abs(Wg))
            du = n_in * oracle.decode(law, q, pos[r], np.abs(x[r]), np.abs(Wu))
            h = oracle.silu(g) * u
            # |silu'| <= 1.1; h is rounded to the call's type once
            dh = 1.1 * dg * np.abs(u) + np.abs(oracle.silu(g)) * du + 8 * 2.0 ** -24 * np.abs(h) + half * np.abs(h)
            wj = w[r, j][:, None]
            y[r] += wj * oracle.decode(law, q, pos[r], h, Wd)
            habs = oracle.decode(law, q, pos[r], np.abs(h), np.abs(Wd))
            err[r] += wj * (oracle.decode(law, q, pos[r], dh, np.abs(Wd)) + (n_out + 64 * 2.0 ** -24) * habs)
            mag[r] += wj * habs
        err += 16 * 2.0 ** -24 * mag
        got = h64(self.y)[rows]
        assert (np.abs(got - y) <= half * np.abs(y) + 1.05 * err + 1e-30).all(), np.abs(got - y).max()


MOE = [
    # B, E, k, D, F, law, q, dtype, pad
    (1, 8, 2, 256, 128, "Q", 1, "bf16", 0),
    (1, 1, 1, 64, 64, "Q", 1, "bf16", 0),          # one expert
    (3, 4, 4, 64, 192, "Q", 2, "bf16", 8),         # every expert chosen, strided rows
    (2, 16, 3, 256, 96, "Q", 2, "bf16", 0),        # 48-column groups
    (9, 8, 2, 256, 512, "Q2xQ2", 4, "bf16", 0),    # two tiles of entries
    (40, 4, 3, 256, 320, "Q2xQ2", 4, "bf16", 16),  # an expert with more entries than a tile
    (64, 24, 5, 512, 256, "Q", 16, "bf16", 0),
    (133, 6, 2, 128, 128, "Q", 8, "bf16", 0),      # two chains of launches
    (5, 60, 6, 416, 208, "Q", 1, "bf16", 0),       # E not a power of two
    (4, 33, 7, 160, 112, "Q", 1, "bf16", 0),       # E off the router's vectors
    (2, 300, 8, 64, 64, "Q", 2, "bf16", 0),        # more than 256 experts
    (2, 2048, 32, 32, 32, "Q", 2, "bf16", 0),      # the limits
    (7, 8, 2, 40, 24, "Q", 2, "bf16", 0),          # groups of 20 and 12: the general path
    (3, 5, 2, 33, 17, "Q", 1, "bf16", 1),          # odd everything
    (1, 4, 2, 64, 96, "Q", 2, "f32", 0),
    (6, 8, 3, 128, 60, "Q2xQ2", 4, "f32", 4),
    (21, 7, 2, 45, 27, "Q", 3, "f32", 0),
    (2, 3, 1, 4096, 64, "Q", 32, "bf16", 0),
    (1, 16, 8, 1024, 768, "Q", 8, "bf16", 0),      # a token: the small clusters
    (32, 64, 8, 1024, 512, "Q", 1, "bf16", 0),     # pieces shared by clusters
    (20, 4, 2, 768, 768, "Q", 1, "bf16", 0),       # two tiles of entries a pass
    (128, 5, 3, 64, 96, "Q", 2, "bf16", 8),        # a full chain, several passes an expert
    (70, 9, 4, 96, 64, "Q", 2, "f32", 0),
    (75, 40, 31, 64, 32, "Q", 2, "bf16", 0),       # chains of 33 entries
    (128, 2048, 8, 32, 16, "Q", 1, "bf16", 0),     # the largest tables
    (128, 2048, 8, 32, 17, "Q", 1, "bf16", 0),
    # pieces of few steps, several a CTA
    (64, 128, 8, 256, 256, "Q", 16, "bf16", 8),
    (32, 128, 32, 256, 256, "Q", 16, "bf16", 0),
    (61, 128, 8, 512, 768, "Q", 8, "bf16", 0),
    (64, 128, 8, 128, 656, "Q", 1, "bf16", 0),
    (33, 100, 8, 64, 1088, "Q2xQ2", 4, "bf16", 16),
    (3, 700, 9, 48, 80, "Q", 1, "f32", 0),         # experts beyond the counted ranking
    (9, 6, 6, 300, 150, "Q", 150, "bf16", 0),      # groups of two and of one
    (5, 12, 3, 202, 62, "Q", 2, "f32", 2),         # vectors off by two
    (1, 2, 2, 512, 512, "Q", 32, "bf16", 0),       # the largest q of the matrix path
    (1, 2, 2, 1024, 512, "Q", 256, "bf16", 0),
]


@gpu
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("B,E,k,D,F,law,q,dtype,pad", MOE)
def test_moe_decode(cuda, B, E, k, D, F, law, q, dtype, pad, renorm):
    m = Moe(B, E, k, D, F, law, q, dtype, seed=B + E + D, pad=pad, residual=renorm)
    m.run(renormalize=renorm)
    assert aal.aal_get_device_status() == aal.AAL_OK
    fast = dtype == "bf16" and q <= 32 and (D // q) % 16 == 0 and (F // q) % 16 == 0 and pad % 8 == 0
    assert aal.aal_last_path() == (aal.AAL_PATH_DECODE if fast else aal.AAL_PATH_GENERAL)
    m.check(renormalize=renorm)
    if pad:
        full = torch.as_strided(m.y, (B, D + pad), (D + pad, 1))
        assert (full[:, D:] == 7.25).all()


@gpu
def test_moe_general_path_on_request(cuda):
    m = Moe(5, 8, 2, 128, 128, "Q", 2, "bf16", seed=3)
    aal.aal_set_path_policy(aal.AAL_PATH_GENERAL)
    try:
        m.run()
        assert aal.aal_last_path() == aal.AAL_PATH_GENERAL
    finally:
        aal.aal_set_path_policy(aal.AAL_PATH_AUTO)
    m.check()
    f = Moe(2, 4, 2, 64, 64, "Q", 2, "f32")
    aal.aal_set_path_policy(aal.AAL_PATH_TENSOR)
    try:
        with pytest.raises(aal.AalError):
            f.run()
    finally:
        aal.aal_set_path_policy(aal.AAL_PATH_AUTO)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_ties_skipped_entries_and_nan(cuda, dtype):
    m = Moe(6, 8, 3, 64, 64, "Q", 2, dtype, seed=8)
    m.Wr[:, 6] = m.Wr[:, 2]       # a tie on every row
    m.Wr[:, 7] = m.Wr[:, 2]
    m.Wr[:, 1] = m.Wr[:, 0]
    m.pos[2] = -5                 # skipped
    m.x[4, 7] = float("nan")      # every logit NaN
    y0, h0 = m.y.clone(), m.h.clone()
    m.run()
    assert aal.aal_get_device_status() == aal.AAL_ERR_DEVICE_BOUNDS
    m.check(rows=np.array([0, 1, 3, 5]))
    assert torch.equal(m.y[2], y0[2]) and torch.equal(m.h[6:9], h0[6:9])
    assert (m.ids[2] == -1).all() and (m.w[2] == 0).all()
    ids = m.ids[4].tolist()
    assert len(set(ids)) == 3 and all(0 <= i < 8 for i in ids)
    assert torch.isnan(m.w[4]).all() and torch.isnan(m.y[4]).all()
    assert aal.aal_get_device_status() == aal.AAL_OK


@gpu
@pytest.mark.parametrize("B", [2, 20])
def test_moe_reads_no_expert_that_was_not_chosen(cuda, B):
    m = Moe(B, 12, 2, 128, 128, "Q", 4, "bf16", seed=5)
    m.Wr[:, 6:] = 0
    m.x[:, 0] = 8.0
    m.Wr[0, :6] = 4.0             # the first six win everywhere
    for t, n in ((m.Wg, m.D), (m.Wu, m.D), (m.Wd, m.F)):
        t[6 * n:] = float("nan")
    m.run()
    assert int(m.ids.max()) < 6 and torch.isfinite(m.y).all()
    m.check()


@gpu
def test_moe_reads_only_the_blocks_of_the_row_type(cuda):
    # one entry of type 1 under Q_4: block (a, k) is used when a is 1 or k
    m = Moe(1, 2, 2, 128, 128, "Q", 4, "bf16", seed=6)
    m.pos[0] = 5
    for t, n in ((m.Wg, 128), (m.Wu, 128), (m.Wd, 128)):
        v = t.view(2, 4, 32, 4, 32)
        for a in range(4):
            for k in range(4):
                if a not in (1, k):
                    v[:, a, :, k] = float("inf")
    m.run()
    assert torch.isfinite(m.y).all()


@gpu
def test_moe_residual_in_place(cuda):
    m = Moe(7, 8, 2, 128, 128, "Q", 2, "bf16", seed=9)
    m.run()
    y = m.y.clone()
    m.y.copy_(m.R)
    m.R = m.y
    m.run()
    assert torch.equal(m.y, y)
    x = m.x.clone()
    m.R, m.y = m.x, m.x           # y = x + experts(x), over x
    m.run()
    got = m.y.clone()
    m.x, m.R, m.y = x, x.clone(), torch.empty_like(x)
    m.run()
    assert torch.equal(got, m.y)


@gpu
def test_norm_then_experts_captured_replayed_and_on_two_streams(cuda):
    """A decode step as it is used: add and norm, then the experts with the
    residual; captured into a graph, replayed on new inputs, and two of them
    side by side on two streams."""
    def make(seed):
        m = Moe(6, 16, 2, 256, 128, "Q", 2, "bf16", seed=seed, residual=False)
        m.hid, m.prev = (torch.randn(6, 256, device="cuda").bfloat16() for _ in range(2))
        m.res = torch.empty_like(m.hid)
        m.gamma = torch.rand(256, device="cuda") + 0.5
        return m

    def step(m, stream=None):
        aal.aal_layer_norm_fwd(m.hid, m.gamma, None, m.x, R=m.prev, S=m.res, stream=stream)
        m.R = m.res
        m.run(stream=stream)

    a, b = make(1), make(2)
    for m in (a, b):
        step(m)
        m.check()
    want = [m.y.clone() for m in (a, b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for m in (a, b):
        m.y.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        step(a, s1)
        step(b, s2)
    torch.cuda.synchronize()
    assert torch.equal(a.y, want[0]) and torch.equal(b.y, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
        step(b)
    for m in (a, b):
        m.hid.copy_(torch.randn(6, 256, device="cuda"))
        m.y.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    got = [m.y.clone() for m in (a, b)]
    for m, y in zip((a, b), got):
        m.check()
        step(m)
        assert torch.equal(m.y, y)


@gpu
def test_layer_norm_bwd_graphs_with_their_own_workspaces(cuda):
    X, dY = (torch.randn(300, 256, device="cuda").bfloat16() for _ in range(2))
    mean, rstd = (torch.from_numpy(v).float().cuda() for v in oracle.layer_norm(h64(X))[1:])
    n = aal.aal_layer_norm_bwd_workspace_size(300, 256)
    graphs, outs = [], []
    for _ in range(2):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dX, dg, db = torch.empty_like(X), torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
        g = torch.cuda.CUDAGraph()
        aal.aal_set_workspace(ws)
        with torch.cuda.graph(g):
            aal.aal_layer_norm_bwd(X, None, mean, rstd, dY, dX=dX, dgamma=dg, dbeta=db)
        aal.aal_set_workspace(None)
        graphs.append((g, ws))
        outs.append((dX, dg, db))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for p, r in zip(*outs):
        assert torch.equal(p, r)
    _, rg, _ = oracle.layer_norm_bwd(h64(X), None, h64(mean), h64(rstd), h64(dY))
    assert oracle.rel_err(h64(outs[0][1]), rg) <= 1e-5


def test_bindings_refuse_wrong_layouts(lib):
    """The compiled marshaller's own checks, on host tensors (nothing launches)."""
    bf = torch.bfloat16
    e = torch.empty(0, 8, dtype=bf)
    with pytest.raises(ValueError, match="unsupported dtype"):
        aal.aal_layer_norm_fwd(e.half(), None, None, e)
    with pytest.raises(ValueError, match="2-D"):
        aal.aal_layer_norm_fwd(torch.empty(0, dtype=bf), None, None, e)
    with pytest.raises(ValueError, match="row-major"):
        aal.aal_layer_norm_fwd(torch.empty(8, 4, dtype=bf).t(), None, None, e)
    with pytest.raises(ValueError, match="overlap"):
        aal.aal_layer_norm_fwd(torch.empty(1, 8, dtype=bf).expand(4, 8), None, None, e)
    with pytest.raises(ValueError, match="contiguous"):
        aal.aal_layer_norm_fwd(e, torch.empty(16, dtype=bf)[::2], None, e)
    with pytest.raises(ValueError, match="contiguous, bf16 or fp32"):
        aal.aal_layer_norm_fwd(e, torch.empty(8, dtype=torch.float16), None, e)
    with pytest.raises(ValueError, match="3 entries|0 entries"):
        aal.aal_layer_norm_fwd(e, None, None, e, rstd=torch.empty(3))
    with pytest.raises((TypeError, AttributeError)):
        aal.aal_layer_norm_fwd(3, None, None, e)
    with pytest.raises(TypeError):
        aal.aal_layer_norm_fwd(e, None, None, e, eps="x")
    with pytest.raises(aal.AalError):
        aal.aal_layer_norm_fwd(e, None, None, e, eps=-1.0)
    w = torch.empty(8, 4, dtype=bf)
    with pytest.raises(ValueError, match="ids"):
        aal.aal_moe_decode("Q", 1, torch.empty(0, dtype=torch.int64), e, w, w, w, w, torch.empty(0, dtype=torch.int32),
                           torch.empty(0), e, e)
    with pytest.raises(ValueError, match="int64"):
        aal.aal_moe_decode("Q", 1, torch.empty(0, dtype=torch.int32), e, e, e, e, e, torch.empty(0, 2, dtype=torch.int32),
                           torch.empty(0, 2), e, e)
    with pytest.raises(KeyError):
        aal.aal_moe_decode("R", 1, torch.empty(0, dtype=torch.int64), e, e, e, e, e, torch.empty(0, 2, dtype=torch.int32),
                           torch.empty(0, 2), e, e)


@gpu
def test_bindings_do_not_take_an_empty_tensor_for_one_left_out(cuda):
    X, Y = (torch.ones(4, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = torch.ones(4, device="cuda")
    none, flat = X[:0], X.reshape(-1)[:0]
    for kw in (dict(R=none), dict(R=X, S=none)):
        with pytest.raises(ValueError, match="no entries"):
            aal.aal_layer_norm_fwd(X, None, None, Y, **kw)
    for g, b in ((flat, None), (None, flat)):
        with pytest.raises(ValueError, match="no entries"):
            aal.aal_layer_norm_fwd(X, g, b, Y)
    for kw in (dict(dX=none), dict(dX=Y, dR=none), dict(dgamma=flat), dict(dbeta=flat)):
        with pytest.raises(ValueError, match="no entries"):
            aal.aal_layer_norm_bwd(X, None, st, st, X, **kw)
    m = Moe(2, 4, 2, 32, 32, "Q", 2, "bf16")
    m.R = m.x[:0]
    with pytest.raises(ValueError, match="no entries"):
        m.run()


FIRST_CALLS_CAPTURED = """
import torch
import associative_algebra_block_b200 as aal

r = lambda *s: torch.randn(*s, device="cuda").bfloat16() * 0.1
X, big = r(64, 768), torch.randn(4, 8192, device="cuda")
mean, rstd = torch.zeros(64, device="cuda"), torch.ones(64, device="cuda")
D, F, E, k, B = 256, 128, 8, 2, 3
pos, ids, w = torch.arange(B, device="cuda"), torch.empty(B, k, dtype=torch.int32, device="cuda"), torch.empty(B, k, device="cuda")
x, Wr, Wg, Wu, Wd, h = r(B, D), r(D, E), r(E * D, F), r(E * D, F), r(E * F, D), r(B * k, F)
Y, dX, bo, dg, y = torch.empty_like(X), torch.empty_like(X), torch.empty_like(big), torch.empty(768, device="cuda"), r(B, D)
ws = torch.empty(aal.aal_layer_norm_bwd_workspace_size(64, 768), dtype=torch.uint8, device="cuda")
aal.aal_set_workspace(ws)

def calls():
    aal.aal_layer_norm_fwd(X, None, None, Y, mean=mean, rstd=rstd)
    aal.aal_layer_norm_fwd(big, None, None, bo)
    aal.aal_layer_norm_bwd(X, None, mean, rstd, Y, dX=dX, dgamma=dg)
    aal.aal_moe_decode("Q", 2, pos, x, Wr, Wg, Wu, Wd, ids, w, h, y)

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (Y, bo, dX, dg, y)]
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (Y, bo, dX, dg, y)))
"""


@gpu
def test_the_first_calls_of_a_process_may_be_captured(cuda):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
