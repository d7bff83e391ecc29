"""Edges of the layer norm and of the experts' step.

Bounds are counted from the arithmetic: U = 2^-24 for a rounding to fp32, half
a step of the output's type (relative 2^-8 for bf16, 2^-24 for fp32) for the
last one."""
from __future__ import annotations

import os
import subprocess
import sys
import threading
import time

import numpy as np
import pytest
import torch

import oracle
import associative_algebra_block_b200 as aal
from test_norm_moe import HALF, TD, Moe, cuda, h64, lib  # noqa: F401 (fixtures)

gpu = pytest.mark.gpu
U = 2.0 ** -24
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------- the experts' general path launches
# A launch may use 48 KB of shared memory, static and dynamic together, unless
# its limit was raised.  These steps' tables need between what the static arrays
# leave of that and 32 KB, in a process that has made no larger call.
FIRST_GENERAL_CALLS = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import associative_algebra_block_b200 as aal
from test_norm_moe import Moe
for n, shape in enumerate({shapes!r}):
    m = Moe(*shape[:-1], seed=n, pad=shape[-1])
    if {captured!r}:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            m.run()
        g.replay()
    else:
        m.run()
    assert aal.aal_get_device_status() == aal.AAL_OK
    assert aal.aal_last_path() == aal.AAL_PATH_GENERAL
    m.check()
"""


def _general_tables(B, E, k):
    """Dynamic shared memory of the general gate/up and down kernels."""
    slots = B * k
    used = min(slots, E)
    passes = min(slots, used + slots // 8)
    up = 16 * passes + 4 * ((2 + (B + 31) // 32) * E + 4 * slots + B)
    up = (up + 15) // 16 * 16
    return up, up + B * 32 * 4


# each process: a step of every form of the kernels (fp32 vectors, fp32 and bf16 by elements)
GENERAL_BANDS = {
    "up and down": [(3, 2048, 8, 32, 24, "Q", 1, "f32", 0), (3, 2048, 8, 34, 22, "Q", 2, "f32", 1),
                    (3, 2048, 8, 33, 17, "Q", 1, "bf16", 0)],
    "down": [(80, 128, 8, 32, 48, "Q", 2, "f32", 0), (90, 24, 8, 30, 26, "Q", 2, "f32", 1),
             (110, 16, 4, 40, 24, "Q", 2, "bf16", 0)],
    "down alone, few experts": [(128, 8, 3, 64, 32, "Q", 1, "f32", 0), (121, 8, 3, 45, 27, "Q", 3, "f32", 0),
                                (128, 8, 3, 40, 24, "Q", 2, "bf16", 0)],
    "up": [(120, 128, 8, 32, 24, "Q", 1, "f32", 0), (128, 128, 8, 27, 33, "Q", 3, "f32", 0),
           (116, 128, 8, 66, 34, "Q", 2, "bf16", 1)],
}


@gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("band", GENERAL_BANDS)
def test_general_experts_launch_as_the_first_calls_of_a_process(cuda, band, captured):
    shapes = GENERAL_BANDS[band]
    for B, E, k, *_ in shapes:
        sizes = _general_tables(B, E, k)
        assert any(22272 < s <= 32768 for s in sizes), sizes
    script = FIRST_GENERAL_CALLS.format(root=ROOT, tests=os.path.join(ROOT, "tests"), shapes=shapes, captured=captured)
    done = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


# ----------------------------------------------------- the backward far from zero
# dx = rstd (g - mean(g) - xh mean(g xh)), every rounding counted:
#   a sum over the row   E = (d / 1024 + 32) u of its terms' magnitudes (a thread's
#                        elements, two trees), and 2 u for the division by d;
#   xh                   2 u (x - mean is rounded against itself, then times rstd)
#                        and as much again within a sum's terms, g u;
#   the three terms      g rstd: 2 u;  rstd mean(g): 3 u;  (x - mean) rstd^2 mean(g xh): 6 u
#                        (in whichever order the factors are taken);
#   their two additions  u of what they add, the first of which counts twice above;
#   then dR, and the output's own rounding.
# Nothing is rounded against x or mean, so the bound does not grow with the offset.
def _bwd_bound(x, mean, rstd, g, ref, d):
    xh = np.abs((x - mean) * rstd)
    e = (d / 1024 + 32) * U
    mg, mgx = np.abs(g).mean(1, keepdims=True), (np.abs(g) * xh).mean(1, keepdims=True)
    return rstd * ((4 * U) * np.abs(g) + (e + 8 * U) * mg + xh * (e + 14 * U) * mgx) + 2 * U * np.abs(ref)


@gpu
@pytest.mark.parametrize("offset", [0.0, 10.0, 100.0, 1000.0, 10000.0])
@pytest.mark.parametrize("m,d,dtype,affine", [
    (300, 40, "f32", "f32"),      # several rows a warp
    (70, 500, "f32", "f32"), (33, 333, "f32", None),
    (64, 1024, "f32", "f32"), (37, 1501, "f32", "f32"), (5, 8192, "f32", "f32"), (3, 5001, "f32", None),
    (3, 9000, "f32", "f32"),      # walked twice
    (65, 768, "bf16", "f32"), (33, 2048, "bf16", "bf16")])
def test_layer_norm_bwd_of_rows_with_an_offset(cuda, m, d, dtype, affine, offset):
    gen = torch.Generator().manual_seed(m + d)
    X = (torch.randn(m, d, generator=gen) + offset).to(TD[dtype])
    x = X.double().numpy()
    mean, rstd = (torch.from_numpy(v).float() for v in oracle.layer_norm(x)[1:])
    mu, rs = mean.double().numpy()[:, None], rstd.double().numpy()[:, None]
    # a gradient that goes with the row: every term of dx counts
    dY = (torch.randn(m, d, generator=gen) + torch.from_numpy((x - mu) * rs)).to(TD[dtype])
    gamma = (torch.randn(d, generator=gen) * 0.1 + 1).to(TD[affine]) if affine else None
    res = m % 2 == 1
    dR = torch.randn(m, d, generator=gen).to(TD[dtype]) if res else None
    dX = torch.full((m, d), float("nan"), dtype=TD[dtype], device="cuda")
    dev = [None if t is None else t.cuda() for t in (X, gamma, mean, rstd, dY, dR)]
    aal.aal_layer_norm_bwd(*dev[:5], dX=dX, dR=dev[5])
    g64 = None if gamma is None else gamma.double().numpy()
    dy = dY.double().numpy()
    ref, _, _ = oracle.layer_norm_bwd(x, g64, mu[:, 0], rs[:, 0], dy)
    err = _bwd_bound(x, mu, rs, dy if gamma is None else dy * g64, ref, d)
    if res:
        ref = ref + dR.double().numpy()
        err = err + U * np.abs(ref)
    assert (np.abs(h64(dX) - ref) <= HALF[dtype] * np.abs(ref) + 1.01 * err).all()


# ------------------------------------------------ the widths that rings hold
@gpu
@pytest.mark.parametrize("d,dtype,affine,one_pass", [
    (8264, "f32", "f32", True), (8268, "f32", "f32", False),
    (14464, "bf16", "f32", True), (14472, "bf16", "f32", False),
    (16384, "bf16", "bf16", True), (16392, "bf16", "bf16", False),
    (8191, "f32", "f32", True), (8193, "f32", "f32", False),    # rows that start anywhere
    (8191, "bf16", "f32", True), (8193, "bf16", "bf16", False)])
def test_layer_norm_bwd_takes_one_pass_up_to_the_stated_widths(cuda, d, dtype, affine, one_pass):
    """On both sides of each width: right, and the workspace used or not."""
    m = 5
    gen = torch.Generator().manual_seed(d)
    X, dY = ((torch.randn(m, d, generator=gen) + s).to(TD[dtype]) for s in (3.0, 0.0))
    gamma = (torch.randn(d, generator=gen) * 0.1 + 1).to(TD[affine])
    x, dy, g64 = X.double().numpy(), dY.double().numpy(), gamma.double().numpy()
    mean, rstd = (torch.from_numpy(v).float() for v in oracle.layer_norm(x)[1:])
    mu, rs = mean.double().numpy()[:, None], rstd.double().numpy()[:, None]
    ws = torch.full((max(256, aal.aal_layer_norm_bwd_workspace_size(m, d)),), 0x5a, dtype=torch.uint8, device="cuda")
    dX = torch.empty(m, d, dtype=TD[dtype], device="cuda")
    dg, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    dev = [t.cuda() for t in (X, gamma, mean, rstd, dY)]
    aal.aal_set_workspace(ws)
    try:
        aal.aal_layer_norm_bwd(*dev, dX=dX, dgamma=dg, dbeta=db)
    finally:
        aal.aal_set_workspace(None)
    assert bool((ws != 0x5a).any()) == one_pass
    ref, rg, rb = oracle.layer_norm_bwd(x, g64, mu[:, 0], rs[:, 0], dy)
    err = _bwd_bound(x, mu, rs, dy * g64, ref, d)
    assert (np.abs(h64(dX) - ref) <= HALF[dtype] * np.abs(ref) + 1.01 * err).all()
    # five rows: at most five additions and as many in the joining sums, xh 2 u
    xh = np.abs((x - mu) * rs)
    assert (np.abs(h64(dg) - rg) <= 13 * U * (np.abs(dy) * xh).sum(0) + U * np.abs(rg)).all()
    assert (np.abs(h64(db) - rb) <= 11 * U * np.abs(dy).sum(0) + U * np.abs(rb)).all()


@gpu
@pytest.mark.parametrize("d,dtype,res", [(14464, "f32", True), (14468, "f32", True), (16384, "f32", False),
                                         (16388, "f32", False), (16384, "bf16", True), (16392, "bf16", True),
                                         (8191, "f32", True), (8193, "f32", True)])
def test_layer_norm_fwd_on_both_sides_of_the_stated_widths(cuda, d, dtype, res):
    m = 5
    gen = torch.Generator().manual_seed(d)
    X, R = (torch.randn(m, d, generator=gen).to(TD[dtype]).cuda() for _ in range(2))
    Y, S = torch.empty_like(X), torch.empty_like(X)
    aal.aal_layer_norm_fwd(X, None, None, Y, R=R if res else None, S=S if res else None)
    s = h64(X) + (h64(R) if res else 0.0)
    ref, mu, rs = oracle.layer_norm(s)
    # a sum: (d / 1024 + 32) u; it enters by the mean, twice by the variance
    big = np.abs(s).max(1)[:, None] * rs[:, None]
    assert (np.abs(h64(Y) - ref) <= HALF[dtype] * np.abs(ref) + 4 * (d / 1024 + 32) * U * big).all()
    if res:
        assert (np.abs(h64(S) - s) <= (HALF[dtype] + U) * np.abs(s)).all()


# ------------------------------------------------------------------ empty widths
def _narrowed(m, D, F):
    """The step with D or F set to 0."""
    m.x, m.Wr, m.y = m.x[:, :D], m.Wr[:D], m.y[:, :D]
    m.Wg, m.Wu, m.Wd, m.h = m.Wg[:m.E * D, :F], m.Wu[:m.E * D, :F], m.Wd[:m.E * F, :D], m.h[:, :F]
    m.D, m.F = D, F
    return m


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("B", [1, 5, 20, 150])
def test_moe_of_width_zero_is_the_residual_and_the_choices(cuda, B, renorm, dtype):
    """F = 0: every expert's product is an empty sum, so y is R (or zero), and
    the router's choices do not depend on F."""
    for residual in (True, False):
        m = _narrowed(Moe(B, 12, 3, 64, 32, "Q", 2, dtype, seed=B, residual=residual), 64, 0)
        if B > 1:
            m.pos[1] = -1  # skipped: its row stays
        m.y.fill_(3.5)
        m.run(renormalize=renorm)
        rows = np.array([b for b in range(B) if b != 1])
        ids, w = oracle.route(h64(m.x)[rows], h64(m.Wr), 3, renorm)
        assert np.array_equal(m.ids.cpu().numpy()[rows], ids)
        assert (np.abs(h64(m.w)[rows] - w) <= 64 * U * w + 1e-38).all()
        want = m.R if residual else torch.zeros_like(m.y)
        assert torch.equal(m.y[rows], want[rows])
        if B > 1:
            assert (m.y[1] == 3.5).all() and (m.ids[1] == -1).all() and (m.w[1] == 0).all()
        assert aal.aal_get_device_status() == (aal.AAL_ERR_DEVICE_BOUNDS if B > 1 else aal.AAL_OK)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_of_inputs_of_width_zero(cuda, dtype):
    """D = 0: every logit is an empty sum, so all tie and the lower indices win;
    h is silu(0) * 0."""
    m = _narrowed(Moe(21, 6, 2, 64, 32, "Q", 2, dtype, residual=False), 0, 32)
    for renorm, weight in ((True, 1 / 2), (False, 1 / 6)):
        m.ids.fill_(-7)
        m.h.fill_(3.5)
        m.run(renormalize=renorm)
        assert m.ids.tolist() == [[0, 1]] * 21 and (m.h == 0).all()
        assert (np.abs(h64(m.w) - weight) <= 64 * U * weight).all()
    assert aal.aal_get_device_status() == aal.AAL_OK


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_of_rows_of_width_zero(cuda, dtype):
    """d = 0: the statistics are those of no element, 0 / 0."""
    X = torch.empty(700, 0, dtype=TD[dtype], device="cuda")
    mean, rstd = torch.zeros(700, device="cuda"), torch.zeros(700, device="cuda")
    aal.aal_layer_norm_fwd(X, None, None, X, R=X, S=X, mean=mean, rstd=rstd)
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()
    aal.aal_layer_norm_fwd(X, None, None, X)
    aal.aal_layer_norm_bwd(X, None, mean, rstd, X, dX=X)
    torch.cuda.synchronize()


# ------------------------------------------------ several rows a warp, many turns
@gpu
@pytest.mark.parametrize("m,d,dtype", [(60001, 8, "bf16"), (40003, 24, "f32"), (30007, 104, "bf16"), (9001, 768, "bf16")])
def test_layer_norm_of_narrow_rows_repeats_itself(cuda, m, d, dtype):
    """A warp refills a stage of its ring once all its rows have left it: the
    same call again, in place and beside another one, gives the same bits."""
    gen = torch.Generator().manual_seed(d)
    X, R = (torch.randn(m, d, generator=gen).to(TD[dtype]).cuda() for _ in range(2))
    Y, S = torch.empty_like(X), torch.empty_like(X)
    aal.aal_layer_norm_fwd(X, None, None, Y, R=R, S=S)
    ref, mu, rs = oracle.layer_norm(h64(X) + h64(R))
    # sums of at most 32 elements a lane and five steps of a tree: (37 + 3) u for
    # the mean against the row's largest element, twice and three times that for
    # the variance's part and the product's
    big = np.abs(h64(X) + h64(R)).max(1)[:, None] * rs[:, None]
    assert (np.abs(h64(Y) - ref) <= HALF[dtype] * np.abs(ref) + 200 * U * big).all()
    other = torch.cuda.Stream()
    A, B = torch.randn(4096, 4096, device="cuda"), torch.empty(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(8):
        with torch.cuda.stream(other):
            aal.aal_layer_norm_fwd(A, None, None, B)
        Xi, Ri = X.clone(), R.clone()
        aal.aal_layer_norm_fwd(Xi, None, None, Ri, R=Ri, S=Xi)
        assert torch.equal(Ri, Y) and torch.equal(Xi, S)
    torch.cuda.synchronize()


# --------------------------------------------------------------------- long steps
@gpu
@pytest.mark.parametrize("B,E,k,D,F,law,q,dtype,pad", [
    (300, 24, 3, 96, 64, "Q", 2, "bf16", 0),     # three chains of launches
    (300, 8, 2, 40, 24, "Q", 2, "bf16", 0),      # the general path
    (257, 16, 4, 64, 48, "Q", 2, "f32", 0)])
def test_moe_of_many_entries(cuda, B, E, k, D, F, law, q, dtype, pad):
    m = Moe(B, E, k, D, F, law, q, dtype, seed=B, pad=pad)
    m.run()
    assert aal.aal_get_device_status() == aal.AAL_OK
    m.check()
    y = m.y.clone()
    for _ in range(5):
        m.y.zero_()
        m.run()
        assert torch.equal(m.y, y)  # the same sums in the same order


# --------------------------------------------------- what a refused launch leaves
# A stream refuses launches once something not allowed in a capture (waiting for
# it) has ended the capture it is in.  The call says so, and the calls after it,
# some of which check their launches by the runtime's last error, are not blamed.
REFUSED_LAUNCH = """
import ctypes
import torch
import associative_algebra_block_b200 as aal

cu = ctypes.CDLL("libcuda.so.1")
X, Y = torch.randn(4, 64, device="cuda"), torch.empty(4, 64, device="cuda")
W, P = torch.randn(64, 32, device="cuda"), torch.empty(4, 32, device="cuda")
pos = torch.arange(4, device="cuda")
s = torch.cuda.Stream()
aal.aal_layer_norm_fwd(X, None, None, Y, stream=s)
aal.aal_decode_matvec("Q", 2, pos, X, W, P)
torch.cuda.synchronize()
want = P.clone()
P.zero_()
torch.cuda.synchronize()
stream, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
assert cu.cuStreamBeginCapture_v2(stream, 2) == 0
assert cu.cuStreamSynchronize(stream) != 0
try:
    aal.aal_layer_norm_fwd(X, None, None, Y, stream=s)
    raise SystemExit("the launch was not refused")
except aal.AalError as e:
    assert e.status == aal.AAL_ERR_CUDA
assert cu.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0
aal.aal_decode_matvec("Q", 2, pos, X, W, P)
torch.cuda.synchronize()
assert torch.equal(P, want)
"""


@gpu
def test_a_refused_launch_leaves_no_error_behind(cuda):
    done = subprocess.run([sys.executable, "-c", REFUSED_LAUNCH], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


# ------------------------------------------------------------------- the binding
SLOW_CALL = r"""
#include <unistd.h>
#include "aal.h"
__attribute__((visibility("default"))) aal_status slow_norm_fwd(aal_mat X, aal_mat R, aal_mat g, aal_mat b, float eps,
    aal_mat S, aal_mat Y, float* m, float* r, void* s) { usleep(400000); return AAL_OK; }
__attribute__((visibility("default"))) aal_status slow_norm_bwd(aal_mat X, aal_mat g, const float* m, const float* r,
    aal_mat dY, aal_mat dR, aal_mat dX, aal_mat dg, aal_mat db, int32_t a, void* s) { usleep(400000); return AAL_OK; }
__attribute__((visibility("default"))) aal_status slow_moe(int32_t law, int32_t q, const int64_t* p, aal_mat x, aal_mat wr,
    aal_mat wg, aal_mat wu, aal_mat wd, aal_mat R, int32_t k, int32_t n, int32_t* i, float* w, aal_mat h, aal_mat y,
    void* s) { usleep(400000); return AAL_OK; }
"""


def test_other_threads_run_while_the_library_is_called(lib, tmp_path, monkeypatch):
    """The marshaller lets go of the interpreter for the call: a full launch
    queue, or a stream that waits for another thread, must not stop that thread."""
    import ctypes
    src, so = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text(SLOW_CALL)
    subprocess.run(["gcc", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-o", str(so), str(src)], check=True)
    slow = ctypes.CDLL(str(so))
    f = aal._fast()
    addr = [ctypes.cast(getattr(slow, n), ctypes.c_void_p).value for n in ("slow_norm_fwd", "slow_norm_bwd", "slow_moe")]
    rest = (torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.cuda.current_device, lambda dev: 0)
    e, z = torch.empty(0, 8), torch.empty(0)
    calls = [lambda: aal.aal_layer_norm_fwd(e, None, None, e),
             lambda: aal.aal_layer_norm_bwd(e, None, z, z, e),
             lambda: aal.aal_moe_decode("Q", 1, torch.empty(0, dtype=torch.int64), e, e, e, e, e,
                                        torch.empty(0, 1, dtype=torch.int32), torch.empty(0, 1), e, e)]
    f.setup(*addr, *rest)
    try:
        for call in calls:
            ticks, stop = [], threading.Event()

            def tick():
                while not stop.is_set():
                    ticks.append(time.monotonic())
                    time.sleep(0.01)

            t = threading.Thread(target=tick)
            t.start()
            t0 = time.monotonic()
            call()
            t1 = time.monotonic()
            stop.set()
            t.join()
            assert t1 - t0 >= 0.3
            # held, the thread would not tick between the call's first and last 0.1 s
            assert any(t0 + 0.1 < v < t1 - 0.1 for v in ticks)
    finally:
        monkeypatch.setattr(aal, "_marshal", None)
        aal._fast()


def test_the_marshaller_is_built_for_this_interpreter(lib):
    """A file built with another interpreter's headers has another name and is
    neither imported nor taken for built."""
    import sysconfig
    from associative_algebra_block_b200 import build
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(build.FASTCALL) == "_fastcall" + suffix
    assert os.path.samefile(aal._fast().__file__, build.FASTCALL)
    assert not os.path.exists(os.path.join(build.PKG, "_fastcall.so"))


def test_every_call_refuses_rows_that_overlap(lib):
    """An expanded row is one row of memory: described as many, a kernel would
    read past it.  (Host tensors: nothing launches.)"""
    bf = torch.bfloat16
    one, X = torch.empty(1, 8, dtype=bf).expand(4, 8), torch.empty(4, 8, dtype=bf)
    for call in (lambda t: aal.mat(t), lambda t: aal.aal_square_product("Q", 2, t, X, X),
                 lambda t: aal.aal_project_fwd("Q", 2, aal.row_rule(seq_len=4), t, X, X),
                 lambda t: aal.aal_layer_norm_fwd(t, None, None, X)):
        with pytest.raises(ValueError, match="overlap"):
            call(one)
        with pytest.raises(ValueError, match="overlap"):
            call(torch.empty(40, dtype=bf).as_strided((4, 8), (3, 1)))
    m = aal.mat(torch.empty(0, 8, dtype=bf))
    assert (m.rows, m.cols, m.ld) == (0, 8, 8)


# --------------------------------------------------------------- calls side by side
@gpu
def test_calls_of_several_threads_at_once(cuda):
    """Four threads, a stream and tensors each, calling at the same time (the
    binding lets them): every one gets what it gets alone."""
    def work(seed):
        gen = torch.Generator().manual_seed(seed)
        shape = [(3, 768), (64, 2048), (5, 1003), (9, 8192)][seed % 4]
        X, dY = (torch.randn(*shape, generator=gen).bfloat16().cuda() for _ in range(2))
        Y, dX = torch.empty_like(X), torch.empty_like(X)
        mean, rstd = torch.empty(shape[0], device="cuda"), torch.empty(shape[0], device="cuda")
        dg = torch.empty(shape[1], device="cuda")
        m = Moe(3 + 30 * seed, 16, 3, 96, 64, "Q", 2, "f32" if seed % 2 else "bf16", seed=seed)
        ws = torch.empty(max(256, aal.aal_layer_norm_bwd_workspace_size(*shape)), dtype=torch.uint8, device="cuda")

        def step():
            aal.aal_set_workspace(ws)
            aal.aal_layer_norm_fwd(X, None, None, Y, mean=mean, rstd=rstd)
            aal.aal_layer_norm_bwd(X, None, mean, rstd, dY, dX=dX, dgamma=dg)
            m.run()
            aal.aal_set_workspace(None)
            return [t.clone() for t in (Y, dX, dg, m.y, m.ids)]
        return step

    steps = [work(s) for s in range(4)]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    wrong = []

    def run(step, expect):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = step()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(g, e) for g, e in zip(got, expect)):
                        wrong.append("differs")
        except Exception as e:  # an assertion here would not reach the test
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=a) for a in zip(steps, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
