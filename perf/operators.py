"""The gated delta rule (prefill and cached step) and the grouped norm with its
gate, as cases to time and to compare: what a serving program holds before each
call (``prepare``), the call itself (``run``: the library's entry points, or the
operators' plain form in elementary float32 tensor operations), what a pass
cannot do without (``work``) and the operators' definitions in float64
(``exact``).

The gated delta rule, per batch row and value head h (key head g = h // (H/G)),
state S (P x N), S = h0 or zeros before the first token:
  dt = softplus(dt_raw + dt_bias_h),  a = exp(-exp(A_log_h) dt),
  beta = sigmoid(b_raw),  k^ = k / sqrt(|k|^2 + 1e-6),  q^ = the same of q
  (k and q as they are without the norm),
  S <- a S (I - beta k^ k^T) + beta v k^T,    y = N^(-1/2) S q^.
Rows of a batch may end early (lengths): tokens behind a row's end change
neither its state nor y.

The grouped norm, channels last: C channels in groups of D, statistics per row
and group, "rms": n = x / sqrt(mean(x^2) + eps), "group": n = (x - mean(x)) /
sqrt(var(x) + eps); out = (n w + bias) SiLU(z), or with the gate before the
norm, the norm of x SiLU(z); without z an activation SiLU(n w + bias), or none.
"""
import math

import torch

own = False

CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    scan = dict(op="scan", io="bf16", N=128, P=128, norm=True, h0=False, ragged=False)
    step = dict(op="step", io="bf16", N=128, P=128, norm=True)
    return [
        # a short prompt on a layer split over several GPUs: few heads, two chunks, latency
        dict(scan, name="scan_prompt", B=1, L=77, G=4, H=8),
        # one prompt on a whole layer: 32 value heads on 16 key heads
        dict(scan, name="scan_layer", B=1, L=4096, G=16, H=32),
        # prompts of different lengths padded to one batch, continuing from cached states
        dict(scan, name="scan_ragged", B=8, L=1000, G=8, H=16, h0=True, ragged=True),
        # a long document on a layer split over two GPUs
        dict(scan, name="scan_long", B=1, L=65536, G=8, H=16),
        # small heads, keys normalised upstream, a length one off the chunk
        dict(scan, name="scan_heads64", B=2, L=2047, G=16, H=16, N=64, P=64, norm=False, h0=True),
        # float32 inputs and outputs, odd length
        dict(scan, name="scan_f32", B=2, L=515, G=4, H=8, N=64, P=128, io="f32"),
        # decode: one sequence, a batch, and float32 with an odd batch
        dict(step, name="step_one", B=1, G=16, H=32),
        dict(step, name="step_batch", B=64, G=16, H=32),
        dict(step, name="step_f32", B=33, G=8, H=8, N=64, P=64, io="f32"),
        # the output norm of a decode step: one norm per head, gate after it
        dict(op="norm", name="norm_decode", io="bf16", rows=64, C=4096, D=128, kind="rms", gate="after"),
        # the same over a long prompt
        dict(op="norm", name="norm_prefill", io="bf16", rows=65536, C=4096, D=128, kind="rms", gate="after"),
        # wide groups with mean and bias, gate before the norm, float32, odd row count
        dict(op="norm", name="norm_groups", io="f32", rows=2047, C=7680, D=1920, kind="group", gate="before"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("scan", "scan", "step", "norm"))
    io = rng.choice(("bf16", "bf16", "f32"))
    N, P = rng.choice((64, 128, 128)), rng.choice((64, 128, 128))
    if op == "scan":
        G = rng.choice((1, 2, 4, 5, 8, 16))
        H = G * rng.choice((1, 2, 4, 5))
        # at most the work of the longest listed prompts: tokens x value heads
        most = (1 << 20) if io == "bf16" else (1 << 14)
        B = min(_log(rng, 1, 16), most // H)
        L = _log(rng, 1, max(1, min(65536, most // (B * H))))
        return dict(op=op, io=io, B=B, L=L, G=G, H=H, N=N, P=P, norm=rng.random() < 0.8,
                    h0=rng.random() < 0.5, ragged=B > 1 and rng.random() < 0.5)
    if op == "step":
        G = rng.choice((1, 2, 4, 8, 16))
        H = G * rng.choice((1, 2, 4))
        return dict(op=op, io=io, B=_log(rng, 1, 2048 // H), G=G, H=H, N=N, P=P, norm=rng.random() < 0.8)
    D = rng.choice((32, 64, 80, 128, 160, 256, 512, 1000, 2048, 4096))
    C = D * rng.choice((1, 2, 5, 8, 16, 32))
    while C > 8192:
        C -= D
    return dict(op=op, io=io, rows=_log(rng, 1, (1 << 27) // C), C=C, D=D, kind=rng.choice(("rms", "group")),
                gate=rng.choice(("after", "before", "act", "none")))


def _lengths(case):
    """Row b's length: from L down to a B-th of it, odd rows one token shorter."""
    B, L = case["B"], case["L"]
    return [max(0, L * (B - b) // B - b % 2) if case["ragged"] else L for b in range(B)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    io = TYPES[case["io"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    if case["op"] == "norm":
        rows, C, D = case["rows"], case["C"], case["D"]
        s = {"case": case, "x": normal(rows, C).to(io), "w": 1.0 + normal(D, std=0.1), "bias": None, "z": None}
        if case["kind"] == "group":
            s["w"], s["bias"] = 1.0 + normal(C, std=0.1), normal(C, std=0.1)
        if case["gate"] in ("after", "before"):
            s["z"] = normal(rows, C).to(io)
        return s
    B, G, H, N, P = (case[k] for k in ("B", "G", "H", "N", "P"))
    T = (case["L"],) if case["op"] == "scan" else ()
    # q, k and v leave a causal convolution with SiLU; the rates start as a trained layer's do
    silu = torch.nn.functional.silu
    q, k, v = silu(normal(B, *T, G, N)), silu(normal(B, *T, G, N)), silu(normal(B, *T, H, P))
    if not case["norm"]:
        q, k = (t / t.norm(dim=-1, keepdim=True).clamp_min(1e-3) for t in (q, k))
    u = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(H, generator=g, device=dev))
    s = {"case": case, "q": q.to(io), "k": k.to(io), "v": v.to(io),
         "dt_raw": normal(B, *T, H, std=math.sqrt(0.5)).to(io), "b_raw": normal(B, *T, H).to(io),
         "params": {"dt_bias": torch.log(torch.expm1(u)),
                    "A_log": torch.log(1.0 + 15.0 * torch.rand(H, generator=g, device=dev))}}
    if case["op"] == "step":
        s["state"] = normal(B, H, P, N, std=0.5)
        return s
    s["h0"] = normal(B, H, P, N, std=0.5) if case["h0"] else None
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev) if case["ragged"] else None
    # where rows end early, y is the program's own buffer: what is behind a row's end stays
    s["y"] = torch.zeros(B, *T, H, P, dtype=io, device=dev) if case["ragged"] else None
    return s


def run(s):
    case = s["case"]
    if own:
        from selective_state_space_52_b200 import axon_ssm
        if case["op"] == "scan":
            out = None if s["y"] is None else (s["y"], torch.empty(case["B"], case["H"], case["P"], case["N"], device=s["v"].device))
            y, h = axon_ssm.delta_scan(s["q"], s["k"], s["v"], s["dt_raw"], s["b_raw"], s["params"], s["h0"],
                                       lengths=s["lengths"], qk_norm=case["norm"], out=out, check=False)
            return {"y": y, "state": h}
        if case["op"] == "step":
            y = axon_ssm.delta_step(s["q"], s["k"], s["v"], s["dt_raw"], s["b_raw"], s["params"], s["state"],
                                    qk_norm=case["norm"])
            return {"y": y, "state": s["state"]}
        return {"y": axon_ssm.gated_norm(s["x"], s["w"], s["z"], bias=s["bias"], group=case["D"], kind=case["kind"],
                                         gate="before" if case["gate"] == "before" else "after",
                                         act=case["gate"] != "none")}
    return {"scan": _scan, "step": _step, "norm": _norm}[case["op"]](s)


# ------------------------------------------------------------ the plain forms
def _rates(s):
    """Log decay (float64: its sums run over many tokens) and beta of every token and value head."""
    x = s["dt_raw"].double() + s["params"]["dt_bias"].double()
    dt = torch.clamp_min(x, 0) + torch.log1p(torch.exp(-x.abs()))
    return -torch.exp(s["params"]["A_log"].double()) * dt, 1 / (1 + torch.exp(-s["b_raw"].float()))


def _keys(s):
    """q (scaled) and k per value head, float32."""
    case = s["case"]
    q, k = s["q"].float(), s["k"].float()
    if case["norm"]:
        q, k = (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    r = case["H"] // case["G"]
    return (q * case["N"] ** -0.5).repeat_interleave(r, -2), k.repeat_interleave(r, -2)


def _step(s):
    q, k = _keys(s)
    g, beta = _rates(s)
    S = s["state"] * torch.exp(g).float()[..., None, None]
    err = beta[..., None] * (s["v"].float() - (S * k[..., None, :]).sum(-1))
    S = S + err[..., None] * k[..., None, :]
    s["state"].copy_(S)
    return {"y": (S * q[..., None, :]).sum(-1).to(s["v"].dtype), "state": s["state"]}


def _scan(s):
    """Chunks of 64 tokens: inside one, with G_i the running log decay,
    (I + A) u = beta (v - e^G k S), A_ij = beta_i e^(G_i - G_j) (k_i . k_j), j < i;
    then y = e^G q S + (q k^T masked and decayed) u, S <- e^G_last S + (e^(G_last - G) u)^T k."""
    case = s["case"]
    B, L, H, N, P = (case[n] for n in ("B", "L", "H", "N", "P"))
    C = CHUNK
    dev = s["v"].device
    q, k = _keys(s)
    g, beta = _rates(s)
    v = s["v"].float()
    ends = torch.tensor(_lengths(case), device=dev)
    live = torch.arange(L, device=dev)[None, :] < ends[:, None]
    if case["ragged"]:
        q, k, v = (torch.where(live[:, :, None, None], t, 0.0) for t in (q, k, v))
        g, beta = (torch.where(live[:, :, None], t, 0.0) for t in (g, beta))
    pad = -L % C
    n = (L + pad) // C

    def chunks(t):
        t = torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, pad))
        return t.reshape(B, n, C, *t.shape[2:]).movedim(3, 1)     # (B, H, n, C, ...)

    q, k, v, g, beta = (chunks(t) for t in (q, k, v, g, beta))
    G = torch.cumsum(g, -1)
    i = torch.arange(C, device=dev)
    below = i[:, None] > i[None, :]
    D = torch.exp(torch.where(i[:, None] >= i[None, :], G[..., :, None] - G[..., None, :], -math.inf)).float()
    A = torch.where(below, beta[..., :, None] * D * (k @ k.transpose(-1, -2)), 0.0)
    T = torch.eye(C, device=dev).expand_as(A).clone()
    for r in range(1, C):                                         # forward substitution, a row of every chunk at once
        T[..., r, :r] = -(A[..., r:r + 1, :r] @ T[..., :r, :r])[..., 0, :]
    T = T * beta[..., None, :]
    M = (q @ k.transpose(-1, -2)) * D
    eG, last = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float()
    end = eG[..., -1]
    ke, qe, kl = k * eG[..., None], q * eG[..., None], k * last[..., None]
    S = torch.zeros(B, H, P, N, device=dev) if s["h0"] is None else s["h0"]
    y = torch.empty(B, H, n, C, P, device=dev)
    for c in range(n):                                            # the state's way from chunk to chunk
        St = S.transpose(-1, -2)
        u = T[:, :, c] @ (v[:, :, c] - ke[:, :, c] @ St)
        y[:, :, c] = qe[:, :, c] @ St + M[:, :, c] @ u
        S = end[:, :, c, None, None] * S + u.transpose(-1, -2) @ kl[:, :, c]
    y = y.movedim(1, 3).reshape(B, n * C, H, P)[:, :L].to(s["v"].dtype)
    if s["y"] is not None:
        s["y"].copy_(torch.where(live[:, :, None, None], y, s["y"]))
        y = s["y"]
    return {"y": y, "state": S}


def _norm(s):
    case = s["case"]
    x = s["x"].float()
    gate = None if s["z"] is None else s["z"].float()
    if gate is not None:
        gate = gate / (1 + torch.exp(-gate))
    if case["gate"] == "before":
        x = x * gate
    n = x.reshape(case["rows"], -1, case["D"])
    if case["kind"] == "group":
        n = n - n.mean(-1, keepdim=True)
    n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + 1e-6)
    if s["bias"] is None:
        o = (n * s["w"]).reshape(case["rows"], -1)
    else:
        o = n.reshape(case["rows"], -1) * s["w"] + s["bias"]
    if case["gate"] == "after":
        o = o * gate
    elif case["gate"] == "act":
        o = o / (1 + torch.exp(-o))
    return {"y": o.to(s["x"].dtype)}


# ------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["C"]
        params = (case["C"] * 2 if case["kind"] == "group" else case["D"]) * 4
        return {"bytes": n * e * (3 if case["gate"] in ("after", "before") else 2) + params, "flops": 8 * n}
    B, G, H, N, P = (case[k] for k in ("B", "G", "H", "N", "P"))
    tokens = sum(_lengths(case)) if case["op"] == "scan" else B
    states = 2 if case["op"] == "step" or case["h0"] else 1
    # per token and value head: S k^, the state's update, S q^, each N P multiply-adds
    return {"bytes": tokens * (2 * G * N + 2 * H * P + 2 * H) * e + B * H * N * P * 4 * states + H * 8,
            "flops": 6 * tokens * H * N * P}


# ------------------------------------------------------------ the definitions in float64
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        rows, C, D = case["rows"], case["C"], case["D"]
        x = s["x"].to(f).view(rows, C // D, D)
        z = None if s["z"] is None else s["z"].to(f).view(rows, C // D, D)
        w, b = s["w"].to(f).view(-1, D), 0.0 if s["bias"] is None else s["bias"].to(f).view(-1, D)
        x = x * z * torch.sigmoid(z) if case["gate"] == "before" else x
        mean = x.mean(-1, keepdim=True) if case["kind"] == "group" else 0.0
        var = (x - mean).pow(2).mean(-1, keepdim=True)
        o = (x - mean) / torch.sqrt(var + 1e-6) * w + b
        o = o * z * torch.sigmoid(z) if case["gate"] == "after" else o * torch.sigmoid(o) if case["gate"] == "act" else o
        return {"y": o.view(rows, C)}
    B, G, H, N, P = (case[k] for k in ("B", "G", "H", "N", "P"))
    L = case["L"] if case["op"] == "scan" else 1
    lens = _lengths(case) if case["op"] == "scan" else [1] * B
    S = s["state"] if case["op"] == "step" else s["h0"]
    S = torch.zeros(B * H, P, N, dtype=f, device="cuda") if S is None else S.to(f).view(B * H, P, N).clone()
    q, k = s["q"].to(f).view(B, L, G, N), s["k"].to(f).view(B, L, G, N)
    if case["norm"]:
        q, k = (t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    head = torch.arange(H, device="cuda") // (H // G)
    a = torch.exp(-torch.exp(s["params"]["A_log"].to(f)) * torch.nn.functional.softplus(
        s["dt_raw"].to(f) + s["params"]["dt_bias"].to(f), threshold=50.0)).view(B, L, H)
    beta = torch.sigmoid(s["b_raw"].to(f)).view(B, L, H)
    v = s["v"].view(B, L, H, P)
    full = min(lens) == L
    y = torch.zeros(B, L, H, P, dtype=f, device="cuda")
    for t in range(L):
        kt, qt = (x[:, t].index_select(1, head).reshape(B * H, N, 1) for x in (k, q))
        d = S * a[:, t].reshape(B * H, 1, 1)
        err = (v[:, t].to(f).reshape(B * H, P, 1) - d @ kt) * beta[:, t].reshape(B * H, 1, 1)
        d = torch.baddbmm(d, err, kt.transpose(1, 2))
        o = (d @ qt).view(B, H, P) * N ** -0.5
        if full:
            S, y[:, t] = d, o
        else:
            alive = torch.tensor([t < e for e in lens], device="cuda")
            S = torch.where(alive.repeat_interleave(H)[:, None, None], d, S)
            y[:, t] = torch.where(alive[:, None, None], o, 0.0)
    S = S.view(B, H, P, N)
    return {"y": y if case["op"] == "scan" else y[:, 0], "state": S}
