"""The state space operators as they are measured: cases, inputs, plain forms and exact values.

The operators follow the short causal convolution in a mixer block:
  scan      selective state space scan of packed prompts, with or without a slot pool of states
  scan_bwd  its gradient (training), with gradients of the initial states where a case has them
  step      one token a sequence against the slot pool
  gated     RMS norm of the scan's output with its gate, by groups of channels
  residual  residual addition with a scale and the RMS norm before the next block

``own`` chooses what ``run`` does: the plain form below (torch, float32) or the package's kernels.
"""
import math

import numpy as np
import torch
import torch.nn.functional as F

own = False

CHUNK = 64  # rows a chunk of the plain scan
EPS = 1e-5


# ------------------------------------------------------------------ cases
def _scan(name, rows, nseq, H, P, G, N, **more):
    return dict(name=name, op="scan", rows=rows, nseq=nseq, H=H, P=P, G=G, N=N, lengths="equal", pool=0, dt32=False) | more


def listed():
    return [
        # serving: a prefill batch of 64 prompts of mixed lengths into a pool of 128 slots
        _scan("scan_prefill_64_prompts_pool", 32512, 64, 64, 64, 4, 128, lengths="mixed", pool=128),
        # serving: one prompt alone, few independent rows of work
        _scan("scan_one_prompt_2048", 2048, 1, 64, 64, 4, 128, pool=4),
        # training: four rows of 4096 tokens, no state kept
        _scan("scan_train_4x4096", 16384, 4, 64, 64, 4, 128),
        # the smallest calls: three short odd prompts, one group, small state
        _scan("scan_short_odd", 97, 3, 24, 48, 1, 40, lengths="mixed", pool=5, dt32=True),
        # training gradient of four rows of 4096 tokens
        _scan("scan_bwd_train_4x4096", 16384, 4, 64, 64, 4, 128) | dict(op="scan_bwd"),
        # training gradient of a shard of packed documents that begins and ends inside documents
        _scan("scan_bwd_packed_states", 2777, 9, 24, 64, 2, 72, lengths="mixed", dt32=True) | dict(op="scan_bwd"),
        # decoding 64 sequences, and a single one with wide heads
        dict(name="step_64_sequences", op="step", nseq=64, H=64, P=64, G=4, N=128, pool=128),
        dict(name="step_one_sequence", op="step", nseq=1, H=32, P=128, G=1, N=64, pool=4),
        # training, forward and backward: the gated norm by groups of 1024 channels
        dict(name="gated_train_16384", op="gated", rows=16384, d=4096, group=1024, first="gate", train=True),
        # decoding: the gated norm of 64 tokens, norm first
        dict(name="gated_decode_64", op="gated", rows=64, d=4096, group=4096, first="norm", train=False),
        # training, forward and backward: residual and norm before a block
        dict(name="residual_train_16384", op="residual", rows=16384, d=2048, res32=True, train=True),
        # decoding: residual and norm, odd width
        dict(name="residual_decode_64_odd", op="residual", rows=64, d=2055, res32=False, train=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_bwd", "scan_bwd", "step", "gated", "residual"])
    if op in ("scan", "scan_bwd"):
        G = rng.choice([1, 2, 4])
        H = G * rng.choice([3, 4, 8, 16])
        nseq = _log(rng, 1, 32)
        P, N = rng.choice([32, 40, 64, 64, 128]), rng.choice([16, 60, 64, 128, 128, 200])
        rows = nseq + min(_log(rng, 30, 12000), 16000 * 64 * 64 * 128 // (H * P * N))
        lengths = rng.choice(["equal", "mixed"])
        rows = rows // nseq * nseq if lengths == "equal" else rows
        return dict(op=op, rows=rows, nseq=nseq, H=H, P=P, G=G, N=N, lengths=lengths,
                    pool=nseq + rng.randrange(4) if op == "scan" and rng.random() < 0.6 else 0, dt32=rng.random() < 0.5)
    if op == "step":
        G = rng.choice([1, 2, 8])
        nseq = _log(rng, 1, 128)
        return dict(op=op, nseq=nseq, H=G * rng.choice([4, 7, 8]), P=rng.choice([32, 52, 64, 128]), G=G,
                    N=rng.choice([16, 64, 100, 128, 256]), pool=nseq + rng.randrange(5))
    rows = _log(rng, 1, 12000)
    if op == "gated":
        group = rng.choice([256, 500, 1024, 2048])
        return dict(op=op, rows=rows, d=group * rng.choice([1, 2]), group=group, first=rng.choice(["gate", "norm"]),
                    train=rng.random() < 0.6)
    return dict(op=op, rows=rows, d=_log(rng, 300, 6000), res32=rng.random() < 0.5, train=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
def _offsets(case, rng):
    n, rows = case["nseq"], case["rows"]
    if case["lengths"] == "equal":
        lens = np.full(n, rows // n)
    else:  # lognormal lengths with the given sum, one token at least
        raw = rng.lognormal(0.0, 1.0, n)
        lens = 1 + np.floor(raw / raw.sum() * (rows - n)).astype(np.int64)
        lens[int(np.argmax(lens))] += rows - int(lens.sum())
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _normal(gen, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _parameters(gen, H):
    """Decay rates in [1, 16], steps around 0.001 .. 0.1 through the bias of softplus, skip weights near one."""
    u = torch.rand(H, generator=gen, device="cuda")
    step = torch.exp(u * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    return dict(A=-(1.0 + 15.0 * torch.rand(H, generator=gen, device="cuda")), D=1.0 + 0.1 * _normal(gen, H, 1.0, torch.float32),
                dt_bias=step + torch.log(-torch.expm1(-step)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    op = case["op"]
    s = dict(case=case, op=op)
    if op in ("scan", "scan_bwd"):
        R, n, H, P, G, N = (case[k] for k in ("rows", "nseq", "H", "P", "G", "N"))
        xbc = F.silu(_normal(gen, (R, H * P + 2 * G * N)))  # the convolution's output row
        s["x"] = xbc[:, :H * P].view(R, H, P)
        s["B"] = xbc[:, H * P:H * P + G * N].view(R, G, N)
        s["C"] = xbc[:, H * P + G * N:].view(R, G, N)
        s["dt"] = _normal(gen, (R, H), 0.5, torch.float32 if case["dt32"] else torch.bfloat16)
        s.update(_parameters(gen, H))
        if case["lengths"] == "equal":
            s["cu"], s["seqlen"] = None, R // n
        else:
            s["cu"], s["seqlen"] = torch.from_numpy(_offsets(case, rng)).cuda(), None
        s["pool"] = s["ci"] = s["hi"] = s["S0"] = s["dS"] = s["dy"] = None
        if case["pool"]:
            s["pool"] = _normal(gen, (case["pool"], H, P, N), 0.5, torch.float32)
            s["ci"] = torch.from_numpy(rng.permutation(case["pool"])[:n].astype(np.int32)).cuda()
            s["hi"] = torch.from_numpy((rng.random(n) < 0.7).astype(np.uint8)).cuda()
        if op == "scan_bwd":
            s["dy"] = _normal(gen, (R, H, P))
            if case["lengths"] == "mixed":
                s["S0"] = _normal(gen, (n, H, P, N), 0.5, torch.float32)
                s["dS"] = _normal(gen, (n, H, P, N), 0.5, torch.float32)
    elif op == "step":
        n, H, P, G, N = (case[k] for k in ("nseq", "H", "P", "G", "N"))
        xbc = F.silu(_normal(gen, (n, H * P + 2 * G * N)))
        s["x"] = xbc[:, :H * P].view(n, H, P)
        s["B"] = xbc[:, H * P:H * P + G * N].view(n, G, N)
        s["C"] = xbc[:, H * P + G * N:].view(n, G, N)
        s["dt"] = _normal(gen, (n, H), 0.5)
        s.update(_parameters(gen, H))
        s["pool"] = _normal(gen, (case["pool"], H, P, N), 0.5, torch.float32)
        s["ci"] = torch.from_numpy(rng.permutation(case["pool"])[:n].astype(np.int32)).cuda()
    else:
        R, d = case["rows"], case["d"]
        s["x"] = _normal(gen, (R, d))
        s["w"] = 1.0 + 0.1 * _normal(gen, (d,), 1.0, torch.float32)
        if op == "gated":
            s["z"] = _normal(gen, (R, d))
        else:
            s["r"] = _normal(gen, (R, d), 2.0, torch.float32 if case["res32"] else torch.bfloat16)
            s["scale"] = 0.22
        if case["train"]:
            s["dy"] = _normal(gen, (R, d))
            if op == "residual":
                s["dr"] = _normal(gen, (R, d), 1.0, s["r"].dtype)
    return s


def work(case):
    op = case["op"]
    if op in ("scan", "scan_bwd"):
        R, n, H, P, G, N = (case[k] for k in ("rows", "nseq", "H", "P", "G", "N"))
        dt = 4 if case["dt32"] else 2
        if op == "scan":
            state = 2 * 4 * n * H * P * N if case["pool"] else 0
            return {"bytes": R * (4 * H * P + 4 * G * N + dt * H) + state,
                    "flops": R * (H * (4 * P * N + CHUNK * P) + G * CHUNK * N)}
        state = 3 * 4 * n * H * P * N if case["lengths"] == "mixed" else 0
        return {"bytes": R * (6 * H * P + 8 * G * N + 2 * dt * H) + state,
                "flops": R * (H * (10 * P * N + 2 * CHUNK * P + 2 * CHUNK * N) + G * CHUNK * N)}
    if op == "step":
        n, H, P, G, N = (case[k] for k in ("nseq", "H", "P", "G", "N"))
        return {"bytes": n * (8 * H * P * N + 4 * H * P + 4 * G * N + 2 * H), "flops": 5 * n * H * P * N}
    R, d = case["rows"], case["d"]
    if op == "gated":  # x, z read, y written; dy, x, z read, dx, dz written
        return {"bytes": R * d * (6 + (10 if case["train"] else 0)), "flops": R * d * (10 + (25 if case["train"] else 0))}
    r = 4 if case["res32"] else 2  # x, r read, y, r' written; dy, dr', r' read, dx, dr written
    return {"bytes": R * d * (4 + 2 * r + (4 + 3 * r if case["train"] else 0)), "flops": R * d * (6 + (15 if case["train"] else 0))}


# ------------------------------------------------------------------ plain forms
def _plain_scan(x, dt, A, B, C, D, dt_bias, cu, seqlen, S0):
    """(y, final states) in float32, by chunks of one sequence each: inside a chunk the masked products, between
    chunks the matrix of decays.  Decay sums are float64.  S0: [nseq, H, P, N]."""
    R, H, P = x.shape
    G, N = B.shape[1:]
    dev = x.device
    if cu is None:
        cu = torch.arange(R // seqlen + 1, device=dev) * seqlen
    cu = cu.long()
    lens = cu[1:] - cu[:-1]
    n = lens.numel()
    ends = torch.cumsum((lens + CHUNK - 1) // CHUNK, 0)  # chunks up to and with each sequence
    count = R // CHUNK + n  # at least the number of chunks
    c = torch.arange(count, device=dev)
    seq = torch.searchsorted(ends, c, right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    first = ends[seq] - (lens[seq] + CHUNK - 1) // CHUNK
    row = (cu[seq] + (c - first) * CHUNK)[:, None] + torch.arange(CHUNK, device=dev)
    valid = (row < cu[seq + 1][:, None]) & real[:, None]
    at = torch.where(valid, row, R)  # a row of zeros for the places past the end

    def chunks(t):
        return F.pad(t, (0, 0) * (t.dim() - 1) + (0, 1))[at]

    dts = dt.double() + dt_bias.double()
    dts = torch.where(dts > 20, dts, torch.log1p(torch.exp(dts.clamp(max=20))))
    xs, Bs, Cs, ds = chunks(x.float()), chunks(B.float()), chunks(C.float()), chunks(dts)
    L = torch.cumsum(ds * A.double(), 1)  # [c, Q, H]
    Lh = L.permute(0, 2, 1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    M = torch.exp((Lh[..., :, None] - Lh[..., None, :]).masked_fill(~lower, -math.inf)).float()  # [c, H, i, j]
    scores = torch.matmul(Cs.permute(0, 2, 1, 3), Bs.permute(0, 2, 3, 1)).repeat_interleave(H // G, 1)
    dh = ds.float().permute(0, 2, 1)
    xh = xs.permute(0, 2, 1, 3)  # [c, H, Q, P]
    Bh = Bs.permute(0, 2, 1, 3).repeat_interleave(H // G, 1)
    Ch = Cs.permute(0, 2, 1, 3).repeat_interleave(H // G, 1)
    y = torch.matmul(scores * M * dh[..., None, :], xh)
    weight = torch.exp(Lh[..., -1:] - Lh).float() * dh
    local = torch.matmul((xh * weight[..., None]).transpose(-1, -2), Bh)  # [c, H, P, N]
    total = torch.cumsum(L[:, -1], 0)  # [c, H]
    before = total - L[:, -1]
    link = (c[:, None] > c) & (seq[:, None] == seq) & real[:, None]
    between = torch.exp((before[:, None] - total).masked_fill(~link[..., None], -math.inf)).float()  # [c, c, H]
    S = torch.matmul(between.permute(2, 0, 1), local.permute(1, 0, 2, 3).reshape(H, count, P * N))
    S = S.reshape(H, count, P, N).transpose(0, 1)
    start = before[first.clamp(max=count - 1)]
    S = S + torch.exp(before - start).float()[..., None, None] * S0[seq]
    y = y + torch.matmul(Ch, S.transpose(-1, -2)) * torch.exp(Lh).float()[..., None]
    y = y + D.float()[:, None, None] * xh
    last = (ends - 1).clamp(min=0)
    final = torch.exp(L[last, -1]).float()[..., None, None] * S[last] + local[last]
    return y.permute(0, 2, 1, 3).reshape(-1, H, P)[torch.argsort(at.reshape(-1), stable=True)[:R]], final


def _initial(s):
    x, n = s["x"], s["case"]["nseq"]
    H, P = x.shape[1:]
    if s["pool"] is not None:
        return s["pool"][s["ci"].long()] * s["hi"][:, None, None, None]
    return s["S0"] if s["S0"] is not None else torch.zeros(n, H, P, s["B"].shape[2], device=x.device)


def _run_scan(s):
    y, final = _plain_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"], s["cu"], s["seqlen"], _initial(s))
    y = y.to(s["x"].dtype)
    if s["pool"] is None:
        return {"y": y}
    s["pool"][s["ci"].long()] = final
    return {"y": y, "pool": s["pool"]}


def _run_scan_bwd(s):
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias")
    leaf = [s[k].detach().to(torch.float32).requires_grad_() for k in names] + [_initial(s).detach().requires_grad_()]
    y, final = _plain_scan(*leaf[:7], s["cu"], s["seqlen"], leaf[7])
    outs, seeds = ([y], [s["dy"].float()]) if s["dS"] is None else ([y, final], [s["dy"].float(), s["dS"]])
    grads = torch.autograd.grad(outs, leaf, seeds)
    out = {"d" + k: g.to(s[k].dtype) for k, g in zip(names, grads)}
    if s["S0"] is not None:
        out["dS0"] = grads[7]
    return out


def _run_step(s):
    heads = s["x"].shape[1] // s["B"].shape[1]
    dt = s["dt"].float() + s["dt_bias"]
    dt = torch.where(dt > 20, dt, torch.log1p(torch.exp(dt.clamp(max=20))))
    x = s["x"].float()
    Bh, Ch = (s[k].float().repeat_interleave(heads, 1) for k in ("B", "C"))
    S = s["pool"][s["ci"].long()]
    S = torch.exp(dt * s["A"])[..., None, None] * S + (dt[..., None] * x)[..., None] * Bh[:, :, None, :]
    y = (S * Ch[:, :, None, :]).sum(-1) + s["D"][:, None] * x
    s["pool"][s["ci"].long()] = S
    return {"y": y.to(s["x"].dtype), "pool": s["pool"]}


def _run_gated(s):
    c = s["case"]
    R, d, g = c["rows"], c["d"], c["group"]
    x, z, w = s["x"].float(), s["z"].float(), s["w"]
    sig = torch.sigmoid(z)
    gate = z * sig
    u = (x * gate if c["first"] == "gate" else x).view(R, d // g, g)
    inv = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    hat = (u * inv).view(R, d)
    y = hat * w if c["first"] == "gate" else hat * w * gate
    out = {"y": y.to(s["x"].dtype)}
    if c["train"]:
        dy = s["dy"].float()
        dn = dy if c["first"] == "gate" else dy * gate
        out["dw"] = (dn * hat).sum(0)
        dh = (dn * w).view(R, d // g, g)
        hv = hat.view(R, d // g, g)
        du = (inv * (dh - hv * (dh * hv).mean(-1, keepdim=True))).view(R, d)
        dgate = du * x if c["first"] == "gate" else dy * hat * w
        out["dx"] = (du * gate if c["first"] == "gate" else du).to(s["x"].dtype)
        out["dz"] = (dgate * sig * (1 + z * (1 - sig))).to(s["z"].dtype)
    return out


def _run_residual(s):
    c = s["case"]
    r = (s["r"].float() + s["scale"] * s["x"].float()).to(s["r"].dtype)
    h = r.float()
    inv = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    hat = h * inv
    out = {"y": (hat * s["w"]).to(s["x"].dtype), "r": r}
    if c["train"]:
        dy = s["dy"].float()
        out["dw"] = (dy * hat).sum(0)
        dh = dy * s["w"]
        dr = inv * (dh - hat * (dh * hat).mean(-1, keepdim=True)) + s["dr"].float()
        out["dx"] = (s["scale"] * dr).to(s["x"].dtype)
        out["dr"] = dr.to(s["r"].dtype)
    return out


# ------------------------------------------------------------------ the package's kernels
def _own(s):
    import causal_depthwise_conv1d_width_amd as cc
    c, op = s["case"], s["op"]
    if op in ("scan", "scan_bwd"):
        args = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"])
        seq = dict(cu_seqlens=s["cu"], seqlen=s["seqlen"])
    if op == "scan":
        if s["pool"] is None:
            return {"y": cc.ssm_scan_fwd(*args, **seq)}
        y = cc.ssm_scan_fwd(*args, **seq, state_pool=s["pool"], cache_indices=s["ci"], has_initial_state=s["hi"])
        return {"y": y, "pool": s["pool"]}
    if op == "scan_bwd":
        g = cc.ssm_scan_bwd(s["dy"], *args, **seq, initial_state=s["S0"], dfinal_state=s["dS"])
        out = {"dx": g.dx, "ddt": g.ddt, "dA": g.dA, "dB": g.dB, "dC": g.dC, "dD": g.dD, "ddt_bias": g.ddt_bias}
        return out if s["S0"] is None else out | {"dS0": g.dinitial_state}
    if op == "step":
        y = cc.ssm_state_update(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"], state_pool=s["pool"],
                                cache_indices=s["ci"])
        return {"y": y, "pool": s["pool"]}
    if op == "gated":
        kw = dict(group_size=c["group"], norm_before_gate=c["first"] == "norm", eps=EPS)
        out = {"y": cc.gated_norm_fwd(s["x"], s["z"], s["w"], **kw)}
        if c["train"]:
            out["dx"], out["dz"], out["dw"] = cc.gated_norm_bwd(s["dy"], s["x"], s["z"], s["w"], **kw)
        return out
    kw = dict(scale=s["scale"], eps=EPS)
    y, r = cc.residual_norm_fwd(s["x"], s["r"], s["w"], **kw)
    out = {"y": y, "r": r}
    if c["train"]:
        out["dx"], out["dr"], out["dw"] = cc.residual_norm_bwd(s["dy"], s["dr"], r, s["w"], **kw)
    return out


def run(state):
    if own:
        return _own(state)
    return {"scan": _run_scan, "scan_bwd": _run_scan_bwd, "step": _run_step, "gated": _run_gated,
            "residual": _run_residual}[state["op"]](state)


# ------------------------------------------------------------------ exact values, from the recurrence in float64
def _softplus64(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def _by_step(s):
    """Inputs laid out [t, sequence, ...] in float64 with the sequences from long to short, and how many are alive at t."""
    R, n = s["case"]["rows"], s["case"]["nseq"]
    cu = np.arange(n + 1) * (R // n) if s["cu"] is None else s["cu"].cpu().numpy().astype(np.int64)
    order = np.argsort(-(cu[1:] - cu[:-1]), kind="stable")
    lens = (cu[1:] - cu[:-1])[order]
    rows = [torch.from_numpy(cu[order][:int((lens > t).sum())] + t).cuda() for t in range(int(lens[0]))]
    return order, rows


def _recur(S, t, rows, v):
    k = rows[t].numel()
    dt, x, Bh = v["dt"][rows[t]], v["x"][rows[t]].double(), v["B"][rows[t]].double().repeat_interleave(v["heads"], 1)
    S = S.clone()
    S[:k] = torch.exp(dt * v["A"])[..., None, None] * S[:k] + (dt[..., None] * x)[..., None] * Bh[:, :, None, :]
    return S


def _exact_scan(s):
    order, rows = _by_step(s)
    v = dict(A=s["A"].double(), dt=_softplus64(s["dt"].double() + s["dt_bias"].double()), x=s["x"], B=s["B"],
             heads=s["x"].shape[1] // s["B"].shape[1])
    S = _initial(s).double()[torch.from_numpy(order).cuda()]
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for t in range(len(rows)):
        k = rows[t].numel()
        S = _recur(S, t, rows, v)
        Ch = s["C"][rows[t]].double().repeat_interleave(v["heads"], 1)
        y[rows[t]] = torch.matmul(S[:k], Ch[..., None])[..., 0] + s["D"].double()[:, None] * s["x"][rows[t]].double()
    if s["pool"] is None:
        return {"y": y}
    pool = s["pool"].double()
    pool[s["ci"].long()[torch.from_numpy(order).cuda()]] = S
    return {"y": y, "pool": pool}


def _exact_scan_bwd(s):
    """Adjoint recurrence, one token at a time; states are kept every 64 steps and made again between them."""
    order, rows = _by_step(s)
    back = torch.from_numpy(np.argsort(order)).cuda()
    at = torch.from_numpy(order).cuda()
    raw = s["dt"].double() + s["dt_bias"].double()
    A, D = s["A"].double(), s["D"].double()
    v = dict(A=A, dt=_softplus64(raw), x=s["x"], B=s["B"], heads=s["x"].shape[1] // s["B"].shape[1])
    G, hg = s["B"].shape[1], v["heads"]
    S = _initial(s).double()[at]
    kept = []
    for t in range(len(rows)):
        if t % 64 == 0:
            kept.append(S)
        S = _recur(S, t, rows, v)
    T = torch.zeros_like(S) if s["dS"] is None else s["dS"].double()[at]
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dB, dC = (torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    dd, dl = (torch.zeros(raw.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in reversed(range(len(kept))):
        states = [kept[b]]
        for t in range(b * 64, min(b * 64 + 64, len(rows))):
            states.append(_recur(states[-1], t, rows, v))
        for t in reversed(range(b * 64, min(b * 64 + 64, len(rows)))):
            r, k = rows[t], rows[t].numel()
            S0, S1 = states[t - b * 64][:k], states[t - b * 64 + 1][:k]
            Bh, Ch = (s[m][r].double().repeat_interleave(hg, 1) for m in ("B", "C"))
            dy, x, d = s["dy"][r].double(), s["x"][r].double(), v["dt"][r]
            T = T.clone()
            T[:k] += dy[..., None] * Ch[:, :, None, :]
            dC[r] = torch.matmul(S1.transpose(-1, -2), dy[..., None])[..., 0].view(k, G, hg, -1).sum(2)
            TB = torch.matmul(T[:k], Bh[..., None])[..., 0]
            dx[r] = d[..., None] * TB + D[:, None] * dy
            dB[r] = (d[..., None] * torch.matmul(T[:k].transpose(-1, -2), x[..., None])[..., 0]).view(k, G, hg, -1).sum(2)
            a = torch.exp(d * A)
            dl[r] = a * (T[:k] * S0).sum((-1, -2))
            dd[r] = dl[r] * A + (x * TB).sum(-1)
            T[:k] *= a[..., None, None]
    ddt = dd * torch.sigmoid(raw)
    out = {"dx": dx, "ddt": ddt, "dA": (dl * v["dt"]).sum(0), "dB": dB, "dC": dC,
           "dD": torch.stack([(s["dy"][:, h].double() * s["x"][:, h].double()).sum() for h in range(A.numel())]),
           "ddt_bias": ddt.sum(0)}
    return out if s["S0"] is None else out | {"dS0": T[back]}


def _exact_step(s):
    v = dict(A=s["A"].double(), dt=_softplus64(s["dt"].double() + s["dt_bias"].double()), x=s["x"], B=s["B"],
             heads=s["x"].shape[1] // s["B"].shape[1])
    pool = s["pool"].double()
    S = _recur(pool[s["ci"].long()], 0, [torch.arange(s["x"].shape[0], device="cuda")], v)
    Ch = s["C"].double().repeat_interleave(v["heads"], 1)
    pool[s["ci"].long()] = S
    return {"y": torch.matmul(S, Ch[..., None])[..., 0] + s["D"].double()[:, None] * s["x"].double(), "pool": pool}


def _exact_norm(s):
    """The norms from their definition, gradients by differentiating it in float64, some rows at a time."""
    c = s["case"]
    R, d = c["rows"], c["d"]
    parts = []
    dw = torch.zeros(d, dtype=torch.float64, device="cuda")
    for a in range(0, R, 2048):
        rows = slice(a, min(R, a + 2048))
        x, w = s["x"][rows].double().requires_grad_(), s["w"].double().requires_grad_()
        o = s["z" if s["op"] == "gated" else "r"][rows].double().requires_grad_()
        if s["op"] == "gated":
            gate = o / (1 + torch.exp(-o))
            u = x * gate if c["first"] == "gate" else x
            v = u.view(u.shape[0], -1, c["group"])
            y = (v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)).view(u.shape) * w
            y = y if c["first"] == "gate" else y * gate
            part = {"y": y}
        else:
            total = (o + s["scale"] * x).detach()
            h = total.to(s["r"].dtype).double().requires_grad_()  # the norm reads the residual as it is stored
            y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * w
            part = {"y": y, "r": total}
        if c["train"] and s["op"] == "gated":
            part["dx"], part["dz"], gw = torch.autograd.grad(y, [x, o, w], s["dy"][rows].double())
            dw += gw
        elif c["train"]:
            gh, gw = torch.autograd.grad(y, [h, w], s["dy"][rows].double())
            part["dr"] = gh + s["dr"][rows].double()
            part["dx"] = s["scale"] * part["dr"]
            dw += gw
        parts.append({k: t.detach() for k, t in part.items()})
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return out | {"dw": dw} if c["train"] else out


def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "scan_bwd": _exact_scan_bwd, "step": _exact_step, "gated": _exact_norm,
            "residual": _exact_norm}[case["op"]](s)
