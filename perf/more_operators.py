"""The gated delta rule's operators, the layer norm and the slots' copies as they are measured: cases, inputs, plain
forms and exact values.

  delta      gated delta rule over packed prompts, with or without a slot pool of states
  delta_bwd  its gradient (training), with gradients of the initial states where a case has them
  update     one token a sequence against the slot pool
  layer      layer norm before a block, alone or of the residual's sum; forward and backward in training
  slots      slots of the pools forked, reordered and cleared in one call

``own`` chooses what ``run`` does: the plain form below (torch, float32) or the package's kernels.
"""
import math

import numpy as np
import torch
import torch.nn.functional as F

own = False

CHUNK = 64  # rows a chunk of the plain form
EPS, NORM_EPS = 1e-5, 1e-6


# ------------------------------------------------------------------ cases
def _delta(name, rows, nseq, H, P, G, N, **more):
    """H value heads of P columns, G key heads of N columns."""
    return dict(name=name, op="delta", rows=rows, nseq=nseq, H=H, P=P, G=G, N=N, lengths="equal", pool=0, f32=False,
                norm=True, beta=1.0) | more


def listed():
    return [
        # serving: a prefill batch of 64 prompts of mixed lengths into a pool of 128 slots
        _delta("delta_prefill_64_prompts_pool", 32512, 64, 32, 128, 16, 128, lengths="mixed", pool=128),
        # serving: one prompt alone, a long chain of few independent rows
        _delta("delta_one_prompt_2048", 2048, 1, 32, 128, 16, 128, pool=4),
        # training: four rows of 4096 tokens, no state kept
        _delta("delta_train_4x4096", 16384, 4, 32, 128, 16, 128),
        # the smallest calls: three short odd prompts, keys as they are, rates up to two
        _delta("delta_short_odd", 97, 3, 6, 48, 2, 40, lengths="mixed", pool=5, f32=True, norm=False, beta=2.0),
        # training gradient of four rows of 4096 tokens
        _delta("delta_bwd_train_4x4096", 16384, 4, 32, 128, 16, 128) | dict(op="delta_bwd"),
        # training gradient of a shard of packed documents that begins and ends inside documents
        _delta("delta_bwd_packed_states", 2777, 9, 12, 64, 4, 72, lengths="mixed", f32=True) | dict(op="delta_bwd"),
        # decoding 64 sequences, and a single one
        dict(name="update_64_sequences", op="update", nseq=64, H=32, P=128, G=16, N=128, pool=128, norm=True, beta=1.0),
        dict(name="update_one_sequence", op="update", nseq=1, H=32, P=64, G=8, N=128, pool=4, norm=True, beta=2.0),
        # training, forward and backward: residual and layer norm before a block
        dict(name="layer_train_16384", op="layer", rows=16384, d=2048, residual="float32", train=True),
        # decoding: the layer norm of 64 tokens, odd width
        dict(name="layer_decode_64_odd", op="layer", rows=64, d=2055, residual="none", train=False),
        # serving: 16 requests of four samples forked, swapped and dropped: convolution and delta states of one layer
        dict(name="slots_reorder_64", op="slots", n=64, slots=128, chan=8192, H=32, P=128, N=128, cleared=8),
        # serving: one short request's states forked to a second slot
        dict(name="slots_fork_one", op="slots", n=1, slots=6, chan=2048, H=8, P=64, N=64, cleared=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_bwd", "delta_bwd", "update", "layer", "slots"])
    if op in ("delta", "delta_bwd"):
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4])
        nseq = _log(rng, 1, 32)
        P, N = rng.choice([32, 40, 64, 128, 128]), rng.choice([16, 60, 64, 128, 128, 200])
        rows = nseq + min(_log(rng, 30, 12000), 16000 * 32 * 128 * 128 // (H * P * N))
        lengths = rng.choice(["equal", "mixed"])
        rows = rows // nseq * nseq if lengths == "equal" else rows
        return dict(op=op, rows=rows, nseq=nseq, H=H, P=P, G=G, N=N, lengths=lengths,
                    pool=nseq + rng.randrange(4) if op == "delta" and rng.random() < 0.6 else 0, f32=rng.random() < 0.5,
                    norm=rng.random() < 0.8, beta=rng.choice([1.0, 2.0]))
    if op == "update":
        G = rng.choice([1, 2, 8])
        nseq = _log(rng, 1, 128)
        return dict(op=op, nseq=nseq, H=G * rng.choice([1, 3, 4]), P=rng.choice([32, 52, 64, 128]), G=G,
                    N=rng.choice([16, 64, 100, 128, 256]), pool=nseq + rng.randrange(5), norm=rng.random() < 0.8,
                    beta=rng.choice([1.0, 2.0]))
    if op == "layer":
        return dict(op=op, rows=_log(rng, 1, 12000), d=_log(rng, 300, 6000),
                    residual=rng.choice(["none", "float32", "bfloat16"]), train=rng.random() < 0.6)
    n = _log(rng, 1, 100)
    return dict(op=op, n=n, slots=n + _log(rng, 1, 64), chan=_log(rng, 200, 6000), H=rng.choice([4, 8, 16]),
                P=rng.choice([40, 64, 128]), N=rng.choice([50, 64, 128]), cleared=rng.randrange(n // 4 + 1))


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
    """Decay rates in [1, 16], steps around 0.001 .. 0.1 through the bias of softplus."""
    u = torch.rand(H, generator=gen, device="cuda")
    step = torch.exp(u * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    return dict(A=-(1.0 + 15.0 * torch.rand(H, generator=gen, device="cuda")), dt_bias=step + torch.log(-torch.expm1(-step)))


def _token_inputs(gen, case, R, dtype):
    """q, k and v side by side in the convolution's output rows; the raw step and rate beside them in the projection's.
    Keys that are not normalised in the call come with a norm near one."""
    H, P, G, N = (case[k] for k in ("H", "P", "G", "N"))
    qkv = F.silu(_normal(gen, (R, 2 * G * N + H * P)))
    if not case["norm"]:
        qkv[:, G * N:2 * G * N] *= 1.2 * N ** -0.5
    return dict(q=qkv[:, :G * N].view(R, G, N), k=qkv[:, G * N:2 * G * N].view(R, G, N), v=qkv[:, 2 * G * N:].view(R, H, P),
                dt=_normal(gen, (R, H), 0.5, dtype), b=_normal(gen, (R, H), 1.0, dtype), **_parameters(gen, H))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    op = case["op"]
    s = dict(case=case, op=op)
    if op in ("delta", "delta_bwd"):
        R, n, H, P, N = (case[k] for k in ("rows", "nseq", "H", "P", "N"))
        s.update(_token_inputs(gen, case, R, torch.float32 if case["f32"] else torch.bfloat16))
        offsets = _offsets(case, rng)
        s["lens"] = np.diff(offsets)  # a scheduler knows its sequences' lengths
        if case["lengths"] == "equal":
            s["cu"], s["seqlen"] = None, R // n
        else:
            s["cu"], s["seqlen"] = torch.from_numpy(offsets).cuda(), None
        s["pool"] = s["ci"] = s["hi"] = s["S0"] = s["dS"] = s["dy"] = None
        if case["pool"]:
            s["pool"] = _normal(gen, (case["pool"], H, P, N), 0.1, torch.float32)
            s["ci"] = torch.from_numpy(rng.permutation(case["pool"])[:n].astype(np.int32)).cuda()
            s["hi"] = torch.from_numpy((rng.random(n) < 0.7).astype(np.uint8)).cuda()
        if op == "delta_bwd":
            s["dy"] = _normal(gen, (R, H, P))
            if case["lengths"] == "mixed":
                s["S0"] = _normal(gen, (n, H, P, N), 0.1, torch.float32)
                s["dS"] = _normal(gen, (n, H, P, N), 0.1, torch.float32)
    elif op == "update":
        n, H, P, N = (case[k] for k in ("nseq", "H", "P", "N"))
        s.update(_token_inputs(gen, case, n, torch.bfloat16))
        s["pool"] = _normal(gen, (case["pool"], H, P, N), 0.1, torch.float32)
        s["ci"] = torch.from_numpy(rng.permutation(case["pool"])[:n].astype(np.int32)).cuda()
    elif op == "layer":
        R, d = case["rows"], case["d"]
        s["x"] = _normal(gen, (R, d))
        s["w"] = 1.0 + 0.1 * _normal(gen, (d,), 1.0, torch.float32)
        s["bias"] = 0.1 * _normal(gen, (d,), 1.0, torch.float32)
        s["r"], s["scale"], s["dr"] = None, 1.0, None
        if case["residual"] != "none":
            dtype = getattr(torch, case["residual"])
            s["r"], s["scale"] = (0.5 + _normal(gen, (R, d), 2.0, torch.float32)).to(dtype), 0.22
            s["dr"] = _normal(gen, (R, d), 1.0, dtype) if case["train"] else None
        if case["train"]:
            s["dy"] = _normal(gen, (R, d))
    else:
        n, slots = case["n"], case["slots"]
        s["conv"] = _normal(gen, (slots, case["chan"], 3))
        s["state"] = _normal(gen, (slots, case["H"], case["P"], case["N"]), 1.0, torch.float32)
        order = rng.permutation(slots)
        target = order[:n]  # distinct; sources come from the same slots, several times over, and from one more
        source = np.concatenate([target[rng.integers(0, n, n - 1)], order[n:n + 1]])
        source[rng.permutation(n)[:case["cleared"]]] = -1
        s["source"], s["target"] = (torch.from_numpy(a.astype(np.int32)).cuda() for a in (source, target))
    return s


def work(case):
    op = case["op"]
    if op in ("delta", "delta_bwd"):
        R, n, H, P, G, N = (case[k] for k in ("rows", "nseq", "H", "P", "G", "N"))
        e = 4 if case["f32"] else 2
        # a chunk: keys' and queries' scores a key head (lower halves); a head, state times keys and queries, the new
        # values, the scores times them, the state's update
        if op == "delta":
            state = 2 * 4 * n * H * P * N if case["pool"] else 0
            return {"bytes": R * (4 * H * P + 4 * G * N + 2 * e * H) + state,
                    "flops": R * (H * (6 * P * N + 2 * CHUNK * P) + G * 2 * CHUNK * N)}
        state = 3 * 4 * n * H * P * N if case["lengths"] == "mixed" else 0
        return {"bytes": R * (6 * H * P + 8 * G * N + 4 * e * H) + state,
                "flops": R * (H * (16 * P * N + 6 * CHUNK * P + 4 * CHUNK * N) + G * 2 * CHUNK * N)}
    if op == "update":
        n, H, P, G, N = (case[k] for k in ("nseq", "H", "P", "G", "N"))
        return {"bytes": n * (8 * H * P * N + 4 * H * P + 4 * G * N + 4 * H), "flops": 7 * n * H * P * N}
    if op == "layer":
        R, d = case["rows"], case["d"]
        r = {"none": 0, "bfloat16": 2, "float32": 4}[case["residual"]]
        forward = 4 + 2 * r  # x (and r) read, y (and r') written
        backward = (4 + 3 * r if r else 6) if case["train"] else 0  # dy, dr', r' read, dx, dr written, or dy, x, dx
        return {"bytes": R * d * (forward + backward), "flops": R * d * (8 + (20 if case["train"] else 0))}
    one = case["chan"] * 3 * 2 + case["H"] * case["P"] * case["N"] * 4
    return {"bytes": (2 * case["n"] - case["cleared"]) * one, "flops": 0}


# ------------------------------------------------------------------ plain forms
def _rate(dt, dt_bias):
    v = dt.double() + dt_bias.double()
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _unit(x, norm):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + NORM_EPS) if norm else x


def _plain_delta(q, k, v, dt, b, A, dt_bias, lens, S0, norm, beta_max):
    """(y, final states) in float32 by chunks of one sequence each; decay sums are float64.  Inside a chunk, with L the
    decays' prefix sums, X = beta_i e^(L_i - L_j) k_i.k_j below the diagonal and S the state before it:
        U = (I + X)^-1 beta (V - e^L K S^T),  Y = scale (e^L Q S^T + (e^(L_i - L_j) q_i.k_j) U),
        S' = e^L_Q S + U^T (e^(L_Q - L) K).   S0: [nseq, H, P, N]."""
    R, H, P = v.shape
    G, N = k.shape[1:]
    dev = v.device
    n = len(lens)
    count = -(-lens // CHUNK)  # chunks of each sequence
    order = np.argsort(-count, kind="stable")  # from long to short: those still running are the first ones
    start = np.concatenate([[0], np.cumsum(lens)])[:-1]
    first = (np.cumsum(count) - count)
    seq = np.repeat(np.arange(n), count)
    row = (start[seq] + (np.arange(len(seq)) - first[seq]) * CHUNK)[:, None] + np.arange(CHUNK)
    at = torch.from_numpy(np.where(row < (start + lens)[seq][:, None], row, R)).to(dev)  # R: a row of zeros

    def chunks(t):
        return F.pad(t, (0, 0) * (t.dim() - 1) + (0, 1))[at]

    hg = H // G
    lc = torch.cumsum(chunks(_rate(dt, dt_bias) * A.double()), 1).transpose(1, 2)  # [c, H, Q]
    beta = (beta_max * chunks(torch.sigmoid(b.float())[..., None])[..., 0]).transpose(1, 2)
    kc, qc = (chunks(_unit(t.float(), norm)).transpose(1, 2) for t in (k, q))  # [c, G, Q, N]
    qc = qc * N ** -0.5
    vc = chunks(v.float()).transpose(1, 2)  # [c, H, Q, P]
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    M = torch.exp((lc[..., :, None] - lc[..., None, :]).masked_fill(~lower, -math.inf)).float()
    kt = kc.transpose(-1, -2)
    X = torch.matmul(kc, kt).repeat_interleave(hg, 1) * M.tril(-1) * beta[..., None]
    scores = torch.matmul(qc, kt).repeat_interleave(hg, 1) * M
    T = torch.eye(CHUNK, device=dev).expand_as(X)
    place = torch.arange(CHUNK, device=dev)
    for level in range(6):  # inverses of diagonal blocks of 2^level rows -> of twice as many
        pair = (place[:, None] >> level) ^ (place >> level)
        T = T - torch.matmul(T, torch.matmul(X * ((pair == 1) & ((place[:, None] >> level) % 2 == 1)), T))
    kc, qc = kc.repeat_interleave(hg, 1), qc.repeat_interleave(hg, 1)
    grow = torch.exp(lc).float()[..., None]
    k_in, q_in = kc * grow, qc * grow
    k_out = kc * torch.exp(lc[..., -1:] - lc).float()[..., None]
    total = torch.exp(lc[..., -1]).float()[..., None, None]
    S = S0[torch.from_numpy(order).to(dev)]
    begins, alive = torch.from_numpy(first[order]).to(dev), [int((count > j).sum()) for j in range(int(count.max(initial=0)))]
    ys, ids = [], []
    for j, m in enumerate(alive):
        c = begins[:m] + j
        Sm = S[:m]
        St = Sm.transpose(-1, -2)
        U = torch.matmul(T[c], beta[c][..., None] * (vc[c] - torch.matmul(k_in[c], St)))
        ys.append(torch.matmul(q_in[c], St) + torch.matmul(scores[c], U))
        ids.append(c)
        S = torch.cat([total[c] * Sm + torch.matmul(U.transpose(-1, -2), k_out[c]), S[m:]])
    y = torch.cat(ys).transpose(1, 2).reshape(-1, H, P)
    y = y[torch.argsort(at[torch.cat(ids)].reshape(-1), stable=True)[:R]]
    return y, S[torch.from_numpy(np.argsort(order)).to(dev)]


def _initial(s):
    H, P = s["v"].shape[1:]
    if s["pool"] is not None:
        return s["pool"][s["ci"].long()] * s["hi"][:, None, None, None]
    return s["S0"] if s["S0"] is not None else torch.zeros(len(s["lens"]), H, P, s["k"].shape[2], device=s["v"].device)


NAMES = ("q", "k", "v", "dt", "b", "A", "dt_bias")


def _run_delta(s):
    c = s["case"]
    y, final = _plain_delta(*(s[m] for m in NAMES), s["lens"], _initial(s), c["norm"], c["beta"])
    y = y.to(s["v"].dtype)
    if s["pool"] is None:
        return {"y": y}
    s["pool"][s["ci"].long()] = final
    return {"y": y, "pool": s["pool"]}


def _run_delta_bwd(s):
    c = s["case"]
    leaf = [s[m].detach().to(torch.float32).requires_grad_() for m in NAMES] + [_initial(s).detach().requires_grad_()]
    y, final = _plain_delta(*leaf[:7], s["lens"], leaf[7], c["norm"], c["beta"])
    outs, seeds = ([y], [s["dy"].float()]) if s["dS"] is None else ([y, final], [s["dy"].float(), s["dS"]])
    grads = torch.autograd.grad(outs, leaf, seeds)
    out = {"d" + m: g.to(s[m].dtype) for m, g in zip(NAMES, grads)}
    return out if s["S0"] is None else out | {"dS0": grads[7]}


def _run_update(s):
    c = s["case"]
    hg, N = s["v"].shape[1] // s["k"].shape[1], s["k"].shape[2]
    beta = c["beta"] * torch.sigmoid(s["b"].float())[..., None]
    q, k = (_unit(s[m].float(), c["norm"]).repeat_interleave(hg, 1)[:, :, None] for m in ("q", "k"))  # [n, H, 1, N]
    decay = torch.exp(_rate(s["dt"], s["dt_bias"]) * s["A"].double()).float()[..., None]
    S = s["pool"][s["ci"].long()]
    u = beta * (s["v"].float() - decay * (S * k).sum(-1))
    S = decay[..., None] * S + u[..., None] * k
    s["pool"][s["ci"].long()] = S
    return {"y": ((S * q).sum(-1) * N ** -0.5).to(s["v"].dtype), "pool": s["pool"]}


def _run_layer(s):
    x, r = s["x"].float(), s["r"]
    stored = x if r is None else (r.float() + s["scale"] * x).to(r.dtype)
    h = stored.float()
    c = h - h.mean(-1, keepdim=True)
    inv = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    hat = c * inv
    out = {"y": (hat * s["w"] + s["bias"]).to(s["x"].dtype)}
    if r is not None:
        out["r"] = stored
    if s["case"]["train"]:
        dy = s["dy"].float()
        out["dw"], out["db"] = (dy * hat).sum(0), dy.sum(0)
        dh = dy * s["w"]
        dr = inv * (dh - dh.mean(-1, keepdim=True) - hat * (dh * hat).mean(-1, keepdim=True))
        if r is not None:
            dr = dr + s["dr"].float()
            out["dr"] = dr.to(r.dtype)
        out["dx"] = (s["scale"] * dr).to(s["x"].dtype)
    return out


def _run_slots(s):
    source, target = s["source"].long(), s["target"].long()
    taken = source >= 0
    for pool in (s["conv"], s["state"]):
        new = pool[source.clamp(min=0)]
        pool[target] = torch.where(taken.view(-1, *[1] * (pool.dim() - 1)), new, torch.zeros_like(new))
    return {"conv": s["conv"], "state": s["state"]}


# ------------------------------------------------------------------ the package's kernels
def _own(s):
    import causal_depthwise_conv1d_width_amd as cc
    c, op = s["case"], s["op"]
    if op in ("delta", "delta_bwd", "update"):
        args = tuple(s[m] for m in NAMES)
        kw = dict(qk_norm=c["norm"], beta_max=c["beta"], norm_eps=NORM_EPS)
    if op in ("delta", "delta_bwd"):
        kw.update(cu_seqlens=s["cu"], seqlen=s["seqlen"])
    if op == "delta":
        if s["pool"] is None:
            return {"y": cc.delta_scan_fwd(*args, **kw)}
        y = cc.delta_scan_fwd(*args, **kw, state_pool=s["pool"], cache_indices=s["ci"], has_initial_state=s["hi"])
        return {"y": y, "pool": s["pool"]}
    if op == "delta_bwd":
        g = cc.delta_scan_bwd(s["dy"], *args, **kw, initial_state=s["S0"], dfinal_state=s["dS"])
        out = {"dq": g.dq, "dk": g.dk, "dv": g.dv, "ddt": g.ddt, "db": g.db, "dA": g.dA, "ddt_bias": g.ddt_bias}
        return out if s["S0"] is None else out | {"dS0": g.dinitial_state}
    if op == "update":
        return {"y": cc.delta_state_update(*args, **kw, state_pool=s["pool"], cache_indices=s["ci"]), "pool": s["pool"]}
    if op == "slots":
        cc.state_copy([s["conv"], s["state"]], s["source"], s["target"])
        return {"conv": s["conv"], "state": s["state"]}
    y, r = cc.layer_norm_fwd(s["x"], s["w"], s["bias"], residual=s["r"], scale=s["scale"], eps=EPS)
    out = {"y": y} if r is None else {"y": y, "r": r}
    if c["train"]:
        if r is None:
            g = cc.layer_norm_bwd(s["dy"], s["x"], s["w"], eps=EPS)
        else:
            g = cc.layer_norm_bwd(s["dy"], r, s["w"], residual=True, dresidual_out=s["dr"], scale=s["scale"], eps=EPS)
            out["dr"] = g.dresidual
        out["dx"], out["dw"], out["db"] = g.dx, g.dweight, g.dbias
    return out


def run(state):
    if own:
        return _own(state)
    return {"delta": _run_delta, "delta_bwd": _run_delta_bwd, "update": _run_update, "layer": _run_layer,
            "slots": _run_slots}[state["op"]](state)


# ------------------------------------------------------------------ exact values, from the recurrence in float64
def _tokens(s):
    """What the recurrence takes, in float64: values, unit keys and queries by head, decays and rates."""
    c = s["case"]
    hg = s["v"].shape[1] // s["k"].shape[1]

    def unit(x):
        x = x.double()
        return (x / torch.sqrt(x.square().sum(-1, keepdim=True) + NORM_EPS) if c["norm"] else x).repeat_interleave(hg, 1)

    raw = s["dt"].double() + s["dt_bias"].double()
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    return dict(q=unit(s["q"]), k=unit(s["k"]), v=s["v"].double(), raw=raw, step=step, a=torch.exp(step * s["A"].double()),
                beta=c["beta"] / (1 + torch.exp(-s["b"].double())), scale=s["k"].shape[2] ** -0.5, hg=hg)


def _token(S, r, t):
    """(state after, prediction S k before the decay, new value u) of rows r; S: [m, H, P, N]."""
    k, a = t["k"][r], t["a"][r][..., None]
    pred = torch.matmul(S, k[..., None])[..., 0]
    u = t["beta"][r][..., None] * (t["v"][r] - a * pred)
    return a[..., None] * S + u[..., None] * k[:, :, None, :], pred, u


def _by_step(s):
    """Sequences from long to short and, for each token position, the rows of those that have it."""
    lens = s["lens"]
    start = np.concatenate([[0], np.cumsum(lens)])[:-1]
    order = np.argsort(-lens, kind="stable")
    rows = [torch.from_numpy(start[order][:int((lens > t).sum())] + t).cuda() for t in range(int(lens.max()))]
    return torch.from_numpy(order).cuda(), rows


def _exact_delta(s):
    order, rows = _by_step(s)
    t = _tokens(s)
    S = _initial(s).double()[order]
    y = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    for r in rows:
        m = r.numel()
        S[:m] = _token(S[:m], r, t)[0]
        y[r] = t["scale"] * torch.matmul(S[:m], t["q"][r][..., None])[..., 0]
    if s["pool"] is None:
        return {"y": y}
    pool = s["pool"].double()
    pool[s["ci"].long()[order]] = S
    return {"y": y, "pool": pool}


def _exact_delta_bwd(s):
    """Adjoint recurrence, one token at a time; states are kept every 64 steps and made again between them."""
    order, rows = _by_step(s)
    t = _tokens(s)
    S = _initial(s).double()[order]
    kept = []
    for j, r in enumerate(rows):
        if j % 64 == 0:
            kept.append(S.clone())
        S[:r.numel()] = _token(S[:r.numel()], r, t)[0]
    T = torch.zeros_like(S) if s["dS"] is None else s["dS"].double()[order]
    dq, dk, dv = (torch.zeros(t[m].shape, dtype=torch.float64, device="cuda") for m in ("q", "k", "v"))
    dl, dbeta = (torch.zeros(t["a"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for c in reversed(range(len(kept))):
        steps = rows[c * 64:c * 64 + 64]
        before = [kept[c]]
        for r in steps:
            m = r.numel()
            before.append(torch.cat([_token(before[-1][:m], r, t)[0], before[-1][m:]]))
        for j in reversed(range(len(steps))):
            r = steps[j]
            m = r.numel()
            S0, Tm = before[j][:m], T[:m]
            S1, pred, u = _token(S0, r, t)
            k, q, a, beta = t["k"][r], t["q"][r], t["a"][r], t["beta"][r]
            dy = t["scale"] * s["dy"][r].double()
            Tm = Tm + dy[..., None] * q[:, :, None, :]
            dq[r] = torch.matmul(S1.transpose(-1, -2), dy[..., None])[..., 0]
            du = torch.matmul(Tm, k[..., None])[..., 0]
            error = t["v"][r] - a[..., None] * pred
            dbeta[r] = (du * error).sum(-1)
            de = beta[..., None] * du
            dv[r] = de
            dk[r] = (torch.matmul(Tm.transpose(-1, -2), u[..., None])
                     - a[..., None, None] * torch.matmul(S0.transpose(-1, -2), de[..., None]))[..., 0]
            Tm = Tm - de[..., None] * k[:, :, None, :]
            dl[r] = a * (Tm * S0).sum((-1, -2))
            T[:m] = a[..., None, None] * Tm

    def through_unit(name, g):
        x = s[name].double()
        g = g.view(*x.shape[:2], t["hg"], -1).sum(2)
        if not s["case"]["norm"]:
            return g
        inv = 1 / torch.sqrt(x.square().sum(-1, keepdim=True) + NORM_EPS)
        return inv * g - inv ** 3 * x * (x * g).sum(-1, keepdim=True)

    ddt = dl * s["A"].double() * torch.sigmoid(t["raw"])
    out = {"dq": through_unit("q", dq), "dk": through_unit("k", dk), "dv": dv, "ddt": ddt,
           "db": dbeta * t["beta"] * (1 - t["beta"] / s["case"]["beta"]), "dA": (dl * t["step"]).sum(0), "ddt_bias": ddt.sum(0)}
    return out if s["S0"] is None else out | {"dS0": T[torch.argsort(order)]}


def _exact_update(s):
    t = _tokens(s)
    pool = s["pool"].double()
    S = _token(pool[s["ci"].long()], torch.arange(s["v"].shape[0], device="cuda"), t)[0]
    pool[s["ci"].long()] = S
    return {"y": t["scale"] * torch.matmul(S, t["q"][..., None])[..., 0], "pool": pool}


def _exact_layer(s):
    """The norm from its definition, gradients by differentiating it in float64, some rows at a time."""
    c = s["case"]
    R, d = c["rows"], c["d"]
    parts, dw, db = [], *(torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2))
    for at in range(0, R, 2048):
        rows = slice(at, min(R, at + 2048))
        total = s["x"][rows].double()
        w, bias = s["w"].double().requires_grad_(), s["bias"].double().requires_grad_()
        if s["r"] is not None:
            total = s["r"][rows].double() + s["scale"] * total
        h = (total if s["r"] is None else total.to(s["r"].dtype).double()).requires_grad_()  # as it is stored
        variance, mean = torch.var_mean(h, -1, correction=0, keepdim=True)
        y = (h - mean) / torch.sqrt(variance + EPS) * w + bias
        part = {"y": y} if s["r"] is None else {"y": y, "r": total}
        if c["train"]:
            gh, gw, gb = torch.autograd.grad(y, [h, w, bias], s["dy"][rows].double())
            if s["r"] is not None:
                gh = gh + s["dr"][rows].double()
                part["dr"] = gh
            part["dx"] = s["scale"] * gh
            dw += gw
            db += gb
        parts.append({m: v.detach() for m, v in part.items()})
    out = {m: torch.cat([p[m] for p in parts]) for m in parts[0]}
    return out | {"dw": dw, "db": db} if c["train"] else out


def _exact_slots(s):
    out = {}
    for name in ("conv", "state"):
        old = s[name].double()
        new = old.clone()
        for a, b in zip(s["source"].tolist(), s["target"].tolist()):
            new[b] = old[a] if a >= 0 else 0.0
        out[name] = new
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "delta_bwd": _exact_delta_bwd, "update": _exact_update, "layer": _exact_layer,
            "slots": _exact_slots}[case["op"]](s)
