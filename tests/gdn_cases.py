"""Seeded inputs and FP64 results of the scalar-gate delta rule for the tests.

The oracle is the repository's per-channel recurrence with the scalar gate
repeated over the channels; dg is then the sum over them."""
import numpy as np
import torch

import oracle
from helpers import DEV
from workloads import round_bf16

NEG = -30000.0


def rnd(dtype, a):
    return round_bf16(a) if dtype == "bf16" else np.ascontiguousarray(a, dtype=np.float32)


def make(seed, lens, *, dtype="bf16", dense=False, H=2, HV=4, K=64, V=64, gate="raw", params=True, l2norm=False,
         h0=True, tail=0, gate_bf16=None, step=(1e-3, 0.3)):
    """lens: sequence lengths (packed), or [T] * B with dense=True. The gate
    spans weak and strong decays; `tail` capacity tokens are NaN."""
    rng = np.random.Generator(np.random.PCG64(seed))
    N, total = len(lens), int(sum(lens))
    B, T = (N, lens[0]) if dense else (1, total + tail)
    n = lambda *s: rng.standard_normal(s, dtype=np.float32)  # noqa: E731
    unit = lambda x: x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), 1e-6)  # noqa: E731
    q, k = n(B, T, H, K), n(B, T, H, K)
    if not l2norm:
        q, k = unit(q), unit(k)
    c = dict(lens=lens, N=N, B=B, T=T, total=total, H=H, HV=HV, K=K, V=V, dtype=dtype, gate_kind=gate,
             l2norm=l2norm, dense=dense, q=rnd(dtype, q), k=rnd(dtype, k), v=rnd(dtype, n(B, T, HV, V)),
             beta=rnd(dtype, 1 / (1 + np.exp(-n(B, T, HV)))), do=rnd(dtype, n(B, T, HV, V)))
    gd = "bf16" if (gate_bf16 if gate_bf16 is not None else dtype == "bf16") else "fp32"
    dt = np.exp(rng.uniform(np.log(step[0]), np.log(step[1]), HV)).astype(np.float32)
    inv = np.log(np.expm1(dt))
    rate = rng.uniform(1, 16, HV).astype(np.float32)
    x = n(B, T, HV)
    c["A_log"] = c["dt_bias"] = None
    if gate == "log":
        x = -rate * np.logaddexp(0, x + inv)
    elif params:
        c["A_log"], c["dt_bias"] = rnd(gd, np.log(rate)), rnd(gd, inv)
    else:
        x = x + inv + np.log(rate)
    c["x"], c["gate_dtype"] = rnd(gd, x.astype(np.float32)), gd
    c["h0"] = 0.1 * n(N, HV, K, V) if h0 else None
    c["dht"] = 0.1 * n(N, HV, K, V) if h0 else None
    c["cu"] = None if dense else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    if tail:
        for m in ("q", "k", "v", "beta", "x", "do"):
            c[m][:, total:] = np.nan
    return c


def natural_gate(c):
    """The natural-log gate [B, T, HV] in FP64."""
    x = c["x"].astype(np.float64)
    if c["gate_kind"] == "log":
        return x
    dt = None if c["dt_bias"] is None else c["dt_bias"][:, None]
    return oracle.gate_activation(x[..., None], c["A_log"], dt)[..., 0]


def _inside(c):
    m = np.zeros((c["B"], c["T"]), bool)
    if c["dense"]:
        m[:] = True
    else:
        m[0, :c["total"]] = True
    return m


def _args(c):
    clean = {m: np.nan_to_num(c[m].astype(np.float64)) for m in ("q", "k", "v", "beta", "do")}
    g = np.nan_to_num(natural_gate(c))
    q, k = clean["q"], clean["k"]
    if c["l2norm"]:
        q, k = oracle.l2norm(q), oracle.l2norm(k)
    return q, k, clean["v"], np.repeat(g[..., None], c["K"], -1), clean["beta"], clean["do"]


def forward(c):
    q, k, v, g, b, _ = _args(c)
    return oracle.recurrence(q, k, v, g, b, c["h0"], c["cu"])


def backward(c):
    q, k, v, g, b, do = _args(c)
    r = oracle.recurrence_bwd(q, k, v, g, b, do, c["h0"], c["dht"], c["cu"])
    dg = r["dg"].sum(-1)
    if c["l2norm"]:
        for m in ("q", "k"):
            y = np.nan_to_num(c[m].astype(np.float64))
            s = np.sqrt((y * y).sum(-1, keepdims=True) + oracle.L2NORM_EPS)
            n = y / s
            r["d" + m] = (r["d" + m] - n * (n * r["d" + m]).sum(-1, keepdims=True)) / s
    r["dA_log"] = r["ddt_bias"] = None
    if c["gate_kind"] == "raw":
        dt = None if c["dt_bias"] is None else c["dt_bias"][:, None]
        dx, dA, db = oracle.gate_activation_bwd(np.nan_to_num(c["x"].astype(np.float64))[..., None], c["A_log"], dt,
                                                dg[..., None], c["cu"])
        r["dg"], r["dA_log"], r["ddt_bias"] = np.nan_to_num(dx[..., 0]), dA, None if db is None else db[:, 0]
    else:
        r["dg"] = dg
    if c["h0"] is None:
        r["dh0"] = None
    return r


def device(c):
    tt = {"bf16": torch.bfloat16, "fp32": torch.float32}
    dev = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(tt[t])  # noqa: E731
    d = {m: dev(c[m], c["dtype"]) for m in ("q", "k", "v", "beta", "do")}
    d.update({m: dev(c[m], c["gate_dtype"]) for m in ("x", "A_log", "dt_bias")})
    d.update({m: dev(c[m], "fp32") for m in ("h0", "dht")})
    d["cu"] = None if c["cu"] is None else torch.from_numpy(c["cu"]).to(DEV)
    return d


def scan_args(d):
    return d["q"], d["k"], d["v"], d["x"], d["beta"], d["h0"]


def scan_kw(c, d):
    return dict(cu_seqlens=d["cu"], use_gate_in_kernel=c["gate_kind"] == "raw", A_log=d["A_log"],
                dt_bias=d["dt_bias"], qk_l2norm=c["l2norm"])


def rel(x, ref, inside=None):
    """Norm of the difference over the norm of the reference (absolute where that is zero)."""
    x = x.detach().double().cpu().numpy() if torch.is_tensor(x) else np.asarray(x, np.float64)
    ref = np.asarray(ref, np.float64)
    if inside is not None:
        x, ref = x[inside], ref[inside]
    assert np.isfinite(x).all()
    n = np.linalg.norm(ref)
    return float(np.linalg.norm(x - ref) / (n if n else 1.0))


def inside(c):
    return _inside(c)
