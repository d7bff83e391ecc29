"""The norm ahead of the feed-forward block and the mixture-of-experts block that follows it at decode time: the
cases that are measured, a plain form of each operator, and its definition in 64 bits.

ln_fwd   layer norm of the rows of X, or of X + R (the residual stream), with the row statistics the backward reads.
ln_bwd   its gradients: dX (with the residual branch's gradient added), dgamma, dbeta.
moe      one new token per entry through a routed mixture of algebraic SwiGLU experts, residual added.

``own`` selects the library's calls; otherwise ``run`` is elementary torch arithmetic in 32 bits (router logits in
64: they decide which expert is taken)."""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def _ln(name, op, rows, d, dtype, residual, affine=None):
    c = {"op": op, "rows": rows, "d": d, "dtype": dtype, "residual": residual, "affine": affine or dtype}
    return dict(c, name=name) if name else c


def _moe(name, batch, experts, top_k, d, f, law, q, dtype):
    c = {"op": "moe", "batch": batch, "experts": experts, "top_k": top_k, "d": d, "f": f, "law": law, "q": q,
         "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token of the 110M pilot, residual added: latency only
        _ln("ln_fwd_token", "ln_fwd", 1, 768, "bf16", True),
        # a training step of the pilot: 8 sequences of 1536, master copies of gamma and beta in fp32
        _ln("ln_fwd_pilot", "ln_fwd", 12288, 768, "bf16", True, "f32"),
        # 2048 tokens of the width-4096 configuration, fp32
        _ln("ln_fwd_wide", "ln_fwd", 2048, 4096, "f32", False),
        # odd width and row count: rows that start anywhere
        _ln("ln_fwd_odd", "ln_fwd", 4099, 1003, "bf16", False),
        # a short fine-tuning batch
        _ln("ln_bwd_small", "ln_bwd", 96, 2048, "bf16", True),
        # the pilot's training step
        _ln("ln_bwd_pilot", "ln_bwd", 12288, 768, "bf16", True, "f32"),
        # the widest configuration, 32768 tokens: the largest norm
        _ln("ln_bwd_large", "ln_bwd", 32768, 5120, "bf16", True),
        # odd width, fp32
        _ln("ln_bwd_odd", "ln_bwd", 2047, 1001, "f32", False),
        # one token through the narrow expert shape under Q_16
        _moe("moe_token", 1, 128, 8, 2048, 768, "Q", 16, "bf16"),
        # a few tokens through dense experts of the same shape (q = 1 is the plain matrix product)
        _moe("moe_dense", 8, 128, 8, 2048, 768, "Q", 1, "bf16"),
        # a serving batch
        _moe("moe_batch", 64, 128, 8, 2048, 768, "Q", 16, "bf16"),
        # the pilot's widths as experts, the tensor-square law, fp32
        _moe("moe_pilot_f32", 5, 8, 2, 768, 1536, "Q2xQ2", 4, "f32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "moe"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op != "moe":
        d = _log_uniform(rng, 48, 8192)
        if rng.random() < 0.7:
            d = max(64, d // 64 * 64)
        rows = min(_log_uniform(rng, 1, 32768), 32768 * 5120 // (2 * d))
        return _ln(None, op, rows, d, dtype, rng.random() < 0.5, rng.choice([dtype, "f32"]))
    law, q = rng.choice([("Q", 1), ("Q", 2), ("Q", 8), ("Q", 16), ("Q2xQ2", 4)])
    d, f = _log_uniform(rng, 256, 2048), _log_uniform(rng, 128, 1536)
    g = rng.choice([q * 16, q * 16, q * 16, q])  # widths off the matrix instruction's grid too
    d, f = max(g, d // g * g), max(g, f // g * g)
    experts = rng.choice([4, 8, 16, 24, 60, 64, 128])
    if dtype == "f32":
        experts = min(experts, 24)
    return _moe(None, _log_uniform(rng, 1, 64), experts, rng.randint(1, min(8, experts)), d, f, law, q, dtype)


# --------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=dt):
        return torch.empty(*shape, dtype=to, device="cuda").normal_(0.0, 1.0, generator=gen).mul_(scale)

    if case["op"] == "moe":
        b, e, d, f = case["batch"], case["experts"], case["d"], case["f"]
        return {"case": case, "kept": {},
                "positions": torch.randint(0, 1536, (b,), generator=gen, device="cuda"),
                "x": normal(b, d), "r": normal(b, d), "wr": normal(d, e, scale=d ** -0.5),
                "wg": normal(e * d, f, scale=d ** -0.5), "wu": normal(e * d, f, scale=d ** -0.5),
                "wd": normal(e * f, d, scale=f ** -0.5)}
    m, d, ft = case["rows"], case["d"], TYPES[case["affine"]]
    # a residual stream's features have offsets and scales of their own
    offset, scale = normal(1, d, to=torch.float32) * 0.5 + 0.25, normal(1, d, to=torch.float32).abs() + 0.5
    st = {"case": case, "kept": {},
          "x": (normal(m, d, to=torch.float32) * scale + offset).to(dt),
          "gamma": (1.0 + 0.1 * normal(d, to=torch.float32)).to(ft), "beta": normal(d, scale=0.1, to=ft)}
    if case["op"] == "ln_fwd":
        st["r"] = normal(m, d) if case["residual"] else None
        return st
    mean, rstd = [], []
    for part in st["x"].split(4096):
        p = part.double()
        mean.append(p.mean(1).float())
        rstd.append((p.var(1, correction=0) + EPS).rsqrt().float())
    st["mean"], st["rstd"] = torch.cat(mean), torch.cat(rstd)
    st["dy"] = normal(m, d)
    st["r"] = normal(m, d) if case["residual"] else None
    return st


def _kept(st, name, *shape, dtype):
    """A buffer that the caller's program keeps from call to call."""
    if name not in st["kept"]:
        st["kept"][name] = torch.empty(*shape, dtype=dtype, device="cuda")
    return st["kept"][name]


# ----------------------------------------------------------------- plain forms
def _plain_ln_fwd(st):
    dt = st["x"].dtype
    s = st["x"].float()
    if st["r"] is not None:
        s = s + st["r"].float()
    mean = s.mean(1, keepdim=True)
    c = s - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    y = c * rstd * st["gamma"].float() + st["beta"].float()
    return {"y": y.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0], "s": s.to(dt) if st["r"] is not None else None}


def _plain_ln_bwd(st):
    dt, ft = st["x"].dtype, st["gamma"].dtype
    rstd, dy = st["rstd"][:, None], st["dy"].float()
    xhat = (st["x"].float() - st["mean"][:, None]) * rstd
    g = dy * st["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if st["r"] is not None:
        dx = dx + st["r"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * xhat).sum(0).to(ft), "dbeta": dy.sum(0).to(ft)}


def _members(law, q, t):
    """[len(t), q, q]: whether group a is a member of S(t, k), indexed [., k, a]."""
    i = torch.arange(q, device=t.device)
    k, a, t = i[:, None], i[None, :], t[:, None, None]
    if law == "Q":
        return (a == t) | (a == k)
    return ((a >> 1 == t >> 1) | (a >> 1 == k >> 1)) & ((a & 1 == t & 1) | (a & 1 == k & 1))


def _typed(x, member):
    """x [n, d] -> [n, q, d]: for output group k the input with the groups outside S(t, k) zeroed."""
    n, q = member.shape[:2]
    return (x.view(n, 1, q, -1) * member[..., None]).reshape(n, q, -1)


def _plain_moe(st):
    c = st["case"]
    b, e, k, d, f, q = c["batch"], c["experts"], c["top_k"], c["d"], c["f"], c["q"]
    logits = st["x"].double() @ st["wr"].double()
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    top = torch.gather(logits, 1, ids).float()
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    member = _members(c["law"], q, st["positions"] % q)
    x = st["x"].float()
    wg, wu, wd = st["wg"].view(e, d, q, f // q), st["wu"].view(e, d, q, f // q), st["wd"].view(e, f, q, d // q)
    if b * k <= e:  # the chosen experts' weights, one copy a choice
        pick, s = ids.reshape(-1), member.repeat_interleave(k, 0)
        xs = _typed(x.repeat_interleave(k, 0), s)
        g = torch.einsum("skd,sdkc->skc", xs, wg[pick].float()).reshape(b * k, f)
        u = torch.einsum("skd,sdkc->skc", xs, wu[pick].float()).reshape(b * k, f)
        h = g / (1.0 + torch.exp(-g)) * u
        out = torch.einsum("skf,sfkc->skc", _typed(h, s), wd[pick].float()).reshape(b, k, d)
    else:  # every expert on every token, then the chosen ones
        xs = _typed(x, member)
        g = torch.einsum("bkd,edkc->ebkc", xs, wg.float()).reshape(e * b, f)
        u = torch.einsum("bkd,edkc->ebkc", xs, wu.float()).reshape(e * b, f)
        h = g / (1.0 + torch.exp(-g)) * u
        hs = _typed(h, member.repeat(e, 1, 1)).view(e, b, q, f)
        out = torch.einsum("ebkf,efkc->bekc", hs, wd.float()).reshape(b, e, d)
        out = torch.gather(out, 1, ids[:, :, None].expand(b, k, d))
    y = st["r"].float() + (w[:, :, None] * out).sum(1)
    return {"y": y.to(st["x"].dtype), "ids": ids.to(torch.int32), "weights": w}


# ------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if not own:
        return {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "moe": _plain_moe}[c["op"]](st)
    import associative_algebra_block_b200 as aal
    dt = st["x"].dtype
    if c["op"] == "ln_fwd":
        m, d = c["rows"], c["d"]
        y = _kept(st, "y", m, d, dtype=dt)
        mean, rstd = _kept(st, "mean", m, dtype=torch.float32), _kept(st, "rstd", m, dtype=torch.float32)
        s = _kept(st, "s", m, d, dtype=dt) if st["r"] is not None else None
        aal.aal_layer_norm_fwd(st["x"], st["gamma"], st["beta"], y, EPS, R=st["r"], S=s, mean=mean, rstd=rstd)
        return {"y": y, "mean": mean, "rstd": rstd, "s": s}
    if c["op"] == "ln_bwd":
        m, d, ft = c["rows"], c["d"], st["gamma"].dtype
        dx = _kept(st, "dx", m, d, dtype=dt)
        dgamma, dbeta = _kept(st, "dgamma", d, dtype=ft), _kept(st, "dbeta", d, dtype=ft)
        if "ws" not in st["kept"]:
            _kept(st, "ws", max(256, aal.aal_layer_norm_bwd_workspace_size(m, d)), dtype=torch.uint8)
        aal.aal_set_workspace(st["kept"]["ws"])
        aal.aal_layer_norm_bwd(st["x"], st["gamma"], st["mean"], st["rstd"], st["dy"], dX=dx, dgamma=dgamma,
                               dbeta=dbeta, dR=st["r"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    b, k = c["batch"], c["top_k"]
    y = _kept(st, "y", b, c["d"], dtype=dt)
    ids, w = _kept(st, "ids", b, k, dtype=torch.int32), _kept(st, "weights", b, k, dtype=torch.float32)
    h = _kept(st, "h", b * k, c["f"], dtype=dt)
    aal.aal_moe_decode(c["law"], c["q"], st["positions"], st["x"], st["wr"], st["wg"], st["wu"], st["wd"], ids, w, h,
                       y, R=st["r"])
    return {"y": y, "ids": ids, "weights": w}


# ----------------------------------------------------------------- lower bounds
def _uses(law, q):
    """For every weight block (a, k), how many of the q row types use it."""
    if law == "Q":
        return [q if a == k else 1 for a in range(q) for k in range(q)]
    pair = {True: 2, False: 1}  # types i with a in S(i, k), per component
    return [pair[a >> 1 == k >> 1] * pair[a & 1 == k & 1] for a in range(q) for k in range(q)]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] != "moe":
        m, d, ft = case["rows"], case["d"], 4 if case["affine"] == "f32" else 2
        if case["op"] == "ln_fwd":  # X (and R) in, Y (and the sum) out, statistics out, gamma and beta
            return {"bytes": m * d * size * (4 if case["residual"] else 2) + 8 * m + 2 * d * ft, "flops": 8 * m * d}
        # X, dY (and the residual's gradient) in, dX out, statistics, gamma in, two gradients out
        return {"bytes": m * d * size * (4 if case["residual"] else 3) + 8 * m + 3 * d * ft, "flops": 14 * m * d}
    b, e, k, d, f, q = (case[n] for n in ("batch", "experts", "top_k", "d", "f", "q"))
    uses = _uses(case["law"], q)
    # with every expert as likely as any other, the expected number of (expert, weight block) pairs some token needs
    blocks = sum(1.0 - (1.0 - k * n / (e * q)) ** b for n in uses) * e
    weights = 3 * d * f / (q * q) * blocks
    return {"bytes": size * (weights + d * e + 3 * b * d) + 8 * b * k + 8 * b,
            "flops": 2 * b * d * e + 2 * b * k * 3 * d * f * sum(uses) / q ** 3}


# --------------------------------------------------------- the definitions, 64 bits
def _in_s(law, t, k, a):
    if law == "Q":
        return a == t if k == t else a in (t, k)
    return _in_s("Q", t // 2, k // 2, a // 2) and _in_s("Q", t % 2, k % 2, a % 2)


def _product(law, q, t, x, w):
    """Row t of the table applied to one row x [din] and w [din, dout], block by block."""
    bi, bo = w.shape[0] // q, w.shape[1] // q
    y = torch.zeros(w.shape[1], dtype=torch.float64, device=w.device)
    for k in range(q):
        for a in range(q):
            if _in_s(law, t, k, a):
                y[k * bo:(k + 1) * bo] += x[a * bi:(a + 1) * bi] @ w[a * bi:(a + 1) * bi, k * bo:(k + 1) * bo]
    return y


def _exact_moe(case, st):
    b, e, k, d, f, q, law = (case[n] for n in ("batch", "experts", "top_k", "d", "f", "q", "law"))
    logits = (st["x"].double() @ st["wr"].double()).cpu()
    ids = [sorted(range(e), key=lambda i: (-row[i], i))[:k] for row in logits.tolist()]
    ids_t = torch.tensor(ids)
    weights = torch.softmax(torch.gather(logits, 1, ids_t), 1).cuda()
    y, x = st["r"].double(), st["x"].double()
    types = (st["positions"] % q).tolist()
    if b * k * q > 1500:  # a row's products through a mask of its type: the same sums in fewer steps
        masks = {}

        def product(t, v, w):
            key = (t, w.shape)
            if key not in masks:
                m = torch.tensor([[float(_in_s(law, t, j, a)) for j in range(q)] for a in range(q)], device="cuda")
                masks[key] = (m.repeat_interleave(w.shape[0] // q, 0).repeat_interleave(w.shape[1] // q, 1)).double()
            return v @ (w * masks[key])
    else:
        def product(t, v, w):
            return _product(law, q, t, v, w)
    for i in range(e):
        rows = [r for r in range(b) if i in ids[r]]
        if not rows:
            continue
        wg, wu = st["wg"][i * d:(i + 1) * d].double(), st["wu"][i * d:(i + 1) * d].double()
        wd = st["wd"][i * f:(i + 1) * f].double()
        for r in rows:
            g, u = product(types[r], x[r], wg), product(types[r], x[r], wu)
            y[r] += weights[r, ids[r].index(i)] * product(types[r], g * torch.sigmoid(g) * u, wd)
    return {"y": y, "ids": ids_t.to(torch.int32), "weights": weights}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "moe":
        return _exact_moe(case, st)
    out = {"y": [], "mean": [], "rstd": [], "s": [], "dx": []}
    m, d = case["rows"], case["d"]
    gamma, beta = st["gamma"].double(), st["beta"].double()
    if case["op"] == "ln_fwd":
        for lo in range(0, m, 4096):
            s = st["x"][lo:lo + 4096].double()
            if case["residual"]:
                s = s + st["r"][lo:lo + 4096].double()
            mu = s.sum(1) / d
            rs = (((s - mu[:, None]) ** 2).sum(1) / d + EPS) ** -0.5
            out["y"].append((s - mu[:, None]) * rs[:, None] * gamma + beta)
            out["mean"].append(mu)
            out["rstd"].append(rs)
            out["s"].append(s)
        got = {n: torch.cat(out[n]) for n in ("y", "mean", "rstd", "s")}
        return got if case["residual"] else dict(got, s=None)
    dgamma = torch.zeros(d, dtype=torch.float64, device="cuda")
    dbeta = torch.zeros(d, dtype=torch.float64, device="cuda")
    for lo in range(0, m, 4096):
        dy, mu, rs = (st[n][lo:lo + 4096].double() for n in ("dy", "mean", "rstd"))
        xh = (st["x"][lo:lo + 4096].double() - mu[:, None]) * rs[:, None]
        dgamma += (dy * xh).sum(0)
        dbeta += dy.sum(0)
        dxh = dy * gamma
        dx = rs[:, None] / d * (d * dxh - dxh.sum(1)[:, None] - xh * (dxh * xh).sum(1)[:, None])
        if case["residual"]:
            dx = dx + st["r"][lo:lo + 4096].double()
        out["dx"].append(dx)
    return {"dx": torch.cat(out["dx"]), "dgamma": dgamma, "dbeta": dbeta}
