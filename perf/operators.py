"""The gated delta rule and the block's fused norms: cases, inputs, plain forms, exact values and work.

Gated delta rule, per value head, with the state S in R^{dv x dk} (a linear fast weight, o = S q):

    S~_t = exp(g_t) S_{t-1},   u_t = beta_t (v_t - S~_t k_t),   S_t = S~_t + u_t k_t^T,   o_t = scale S_t q_t

with q and k L2-normalised per token and head, value heads sharing the query/key heads in order.  It is
taken over whole packed sequences (forward and backward) and over one token of many sequences.

Block norms, per row of D values:

    p = RMSNorm(y) w_post SiLU(z)    (the mean over D, or over groups of `group` columns that share w_post)
    x' = x + lambda p,   n = RMSNorm(x') w_pre

and its backward pass.  x, z, n and the weights can be left out.
"""
import math

import torch

own = False
EPS = 1e-6
CHUNK = 64


# --------------------------------------------------------------------------- cases


def _delta(name, kind, lens, hk, hv, dk, dv, dtype="bf16", packed=False, s0=True):
    return {"name": name, "kind": kind, "lens": ",".join(map(str, lens)), "hk": hk, "hv": hv, "dk": dk, "dv": dv,
            "dtype": dtype, "packed": packed, "s0": s0}


def listed():
    ragged = [0, 1, 63, 64, 65, 127, 333, 1000, 17, 2049, 4096, 129, 700, 1374, 255, 3000]
    return [
        # two short sequences of the framework's smallest layer, in fp32
        _delta("delta_fwd_fp32_tiny", "delta_fwd", [64, 64], 1, 1, 64, 64, dtype="fp32"),
        # one frame of a token stream through 4 heads of 192, with the state carried from the frame before
        _delta("delta_fwd_frame", "delta_fwd", [1374], 4, 4, 192, 192),
        # a serving prefill: packed prompts of very different lengths, empty ones among them, q, k and v as
        # slices of one projection, two value heads to a query/key head
        _delta("delta_fwd_packed", "delta_fwd", ragged, 8, 16, 128, 128, packed=True),
        # one long chunk of a causal stream, few heads: the sequence is the only long axis
        _delta("delta_fwd_long", "delta_fwd", [131072], 4, 4, 192, 192),
        # a training microbatch: 8 packed documents, no carried state
        _delta("delta_bwd_packed", "delta_bwd", [1024, 2048, 511, 1, 1500, 77, 1883, 1148], 8, 16, 128, 128,
               packed=True, s0=False),
        # training on one long document, with the gradient into the state that it starts from
        _delta("delta_bwd_long", "delta_bwd", [32768], 4, 4, 192, 192),
        # decoding: one sequence, where the launch is what counts
        {"name": "delta_step_one", "kind": "delta_step", "batch": 1, "slots": 8, "hk": 4, "hv": 4, "dk": 192,
         "dv": 192, "dtype": "bf16"},
        # decoding: a full batch over a pool of states, some rows padding
        {"name": "delta_step_batch", "kind": "delta_step", "batch": 250, "slots": 300, "hk": 8, "hv": 16, "dk": 128,
         "dv": 128, "dtype": "bf16"},
        # a decode step's norms in fp32
        {"name": "norm_fwd_few_fp32", "kind": "norm_fwd", "rows": 7, "D": 768, "group": 768, "dtype": "fp32",
         "residual": True, "gate": True},
        # a prefill's norms
        {"name": "norm_fwd_rows", "kind": "norm_fwd", "rows": 131072, "D": 768, "group": 768, "dtype": "bf16",
         "residual": True, "gate": True},
        # training: the gated norm of each head's outputs for one frame (4 heads share the weight)
        {"name": "norm_bwd_heads", "kind": "norm_bwd", "rows": 1374, "D": 768, "group": 192, "dtype": "bf16",
         "residual": False, "gate": True},
        # training: a large microbatch of a wide block
        {"name": "norm_bwd_rows", "kind": "norm_bwd", "rows": 65536, "D": 2048, "group": 2048, "dtype": "bf16",
         "residual": True, "gate": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["delta_fwd", "delta_bwd", "delta_step", "norm_fwd", "norm_bwd"])
    if kind.startswith("delta"):
        dk = rng.choice([64, 128, 192, 64, 128, 192, 256, 80, 96, 40])
        dv = rng.choice([dk, dk, 64, 128, 192, 256, 72, 16])
        hk = rng.choice([1, 2, 3, 4, 8])
        hv = hk * rng.choice([1, 1, 2, 3])
        if kind == "delta_step":
            batch = _log_int(rng, 1, 512)
            return {"kind": kind, "batch": batch, "slots": batch + rng.randint(1, 40), "hk": hk, "hv": hv, "dk": dk,
                    "dv": dv, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"]) if kind == "delta_fwd" else "bf16"
        most = 2048 if dtype == "fp32" else 32768 if kind == "delta_fwd" else 8192
        total = min(_log_int(rng, 1, most), int(most * 4 * 192 * 192 / (hv * dk * dv)) + 1)
        n = min(_log_int(rng, 1, 24), total)
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        c = _delta("", kind, lens, hk, hv, dk, dv, dtype=dtype, packed=rng.random() < 0.5, s0=rng.random() < 0.6)
        del c["name"]
        return c
    group = rng.choice([64, 128, 192, 96, 80])
    D = rng.choice([group * rng.randint(1, 16), rng.choice([768, 1024, 2048, 1000, 4096, 777, 8192])])
    if D % group or rng.random() < 0.6:
        group = D
    rows = min(_log_int(rng, 1, 65536), 65536 * 2048 // D)
    return {"kind": kind, "rows": rows, "D": D, "group": group, "dtype": rng.choice(["bf16", "bf16", "fp32"]),
            "residual": rng.random() < 0.7, "gate": rng.random() < 0.7}


# --------------------------------------------------------------------------- inputs


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _tokens(case, rows, gen, packed):
    """q, k, v [rows][heads * d]: separate, or columns of one projection's rows."""
    nq, nv = case["hk"] * case["dk"], case["hv"] * case["dv"]
    x = torch.randn((rows, 2 * nq + nv), generator=gen, device="cuda").to(_dt(case))
    parts = x[:, :nq], x[:, nq:2 * nq], x[:, 2 * nq:]
    return parts if packed else tuple(p.contiguous() for p in parts)


def _gates(rows, hv, gen):
    """Log decay -a softplus(x + b) with a in [1, 16], softplus(b) in [0.001, 0.1], and beta = sigmoid(x)."""
    r = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    a = torch.exp(r(hv) * math.log(16.0))
    dt = torch.exp(math.log(0.001) + r(hv) * math.log(100.0))
    b = torch.log(torch.expm1(dt))
    g = -a * torch.nn.functional.softplus(n(rows, hv) + b)
    return g.contiguous(), torch.sigmoid(n(rows, hv)).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dt(case)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    st = dict(case)
    if case["kind"].startswith("delta"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        st["scale"] = dk ** -0.5
        if case["kind"] == "delta_step":
            B, n = case["batch"], case["slots"]
            st["q"], st["k"], st["v"] = _tokens(case, B, gen, False)
            st["g"], st["beta"] = _gates(B, hv, gen)
            st["S"] = rn(n, hv, dv, dk) * 0.3
            slots = torch.randperm(n, generator=gen, device="cuda")[:B].to(torch.int32)
            if B > 8:
                slots[B - B // 16:] = -1  # the batch's padding
            st["slot"] = slots
            st["o"] = torch.zeros((B, hv * dv), dtype=dt, device="cuda")
        else:
            lens = _lens(case)
            T, N = sum(lens), len(lens)
            st["T"], st["N"], st["lens_list"] = T, N, lens
            st["q"], st["k"], st["v"] = _tokens(case, T, gen, case["packed"])
            st["g"], st["beta"] = _gates(T, hv, gen)
            st["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device="cuda")
            st["S0"] = rn(N, hv, dv, dk) * 0.3 if case["s0"] else None
            if case["kind"] == "delta_fwd":
                st["o"] = torch.zeros((T, hv * dv), dtype=dt, device="cuda")
                st["S"] = torch.zeros((N, hv, dv, dk), device="cuda")
            else:
                st["do"] = rn(T, hv * dv).to(dt)
                st["dS"] = rn(N, hv, dv, dk) * 0.3 if case["s0"] else None
    else:
        R, D, G = case["rows"], case["D"], case["group"]
        st["y"] = (rn(R, D) * 2.0).to(dt)
        st["x"] = rn(R, D).to(dt) if case["residual"] else None
        st["z"] = rn(R, D).to(dt) if case["gate"] else None
        st["w_post"] = 1.0 + 0.2 * rn(G)
        st["lam"] = 0.5 + 0.1 * rn(D) if case["residual"] else None
        st["w_pre"] = 1.0 + 0.2 * rn(D) if case["residual"] else None
        if case["kind"] == "norm_bwd":
            st["dxo"] = rn(R, D).to(dt)
            st["dn"] = rn(R, D).to(dt) if case["residual"] else None
    if own:
        _plan(st)
    return st


# --------------------------------------------------------------------------- the framework's calls


def _plan(st):
    """What a program that uses the framework keeps: dims, strides, workspaces and output buffers."""
    from test_weight_layers_b200 import ttt as T
    dt = T.dtype_code(st["q"].dtype if "q" in st else st["y"].dtype)
    if st["kind"].startswith("delta"):
        st["dm"] = T.delta_dims(st["hk"], st["hv"], st["dk"], st["dv"])
        if st["kind"] != "delta_step":
            st["io"] = T.io_cfg(ld_q=st["q"].stride(0), ld_k=st["k"].stride(0), ld_v=st["v"].stride(0))
            back = st["kind"] == "delta_bwd"
            st["ws"] = T.delta_workspace(st["dm"], st["T"], st["N"], dt, backward=back)
            if back:
                st["dq"], st["dk_"], st["dv_"] = (torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
                                                  if not st["packed"] else None for t in (st["q"], st["k"], st["v"]))
                if st["packed"]:  # gradients as slices of one buffer, as the projection's backward takes them
                    nq, nv = st["hk"] * st["dk"], st["hv"] * st["dv"]
                    b = torch.empty((st["T"], 2 * nq + nv), dtype=st["q"].dtype, device="cuda")
                    st["dq"], st["dk_"], st["dv_"] = b[:, :nq], b[:, nq:2 * nq], b[:, 2 * nq:]
                st["dg"], st["dbeta"] = torch.empty_like(st["g"]), torch.empty_like(st["beta"])
                st["dS0"] = torch.empty_like(st["S0"]) if st["s0"] else None
        else:
            st["io"] = T.io_cfg()
    else:
        st["cfg"] = T.norm_cfg(st["D"], st["group"], EPS)
        e = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
        if st["kind"] == "norm_fwd":
            st["xo"], st["n"] = torch.empty_like(st["y"]), e(st["x"])
        else:
            st["ws"] = T.norm_workspace(st["rows"], st["cfg"])
            st["dy"], st["dx"], st["dz"] = torch.empty_like(st["y"]), e(st["x"]), e(st["z"])
            st["dw_post"], st["dlam"], st["dw_pre"] = e(st["w_post"]), e(st["lam"]), e(st["w_pre"])


def _own(st):
    from test_weight_layers_b200 import ttt as T
    kind = st["kind"]
    if kind == "delta_fwd":
        T.ttt_delta_chunked(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"], st["S"], st["o"], st["T"],
                            st["dm"], st["io"], st["ws"], cu_seqlens=st["cu"], n_seq=st["N"], scale=st["scale"])
        return {"o": st["o"], "S": st["S"]}
    if kind == "delta_bwd":
        T.ttt_delta_chunked_backward(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"], st["do"], st["dS"],
                                     st["dq"], st["dk_"], st["dv_"], st["dg"], st["dbeta"], st["dS0"], st["T"],
                                     st["dm"], st["io"], st["ws"], cu_seqlens=st["cu"], n_seq=st["N"],
                                     scale=st["scale"])
        return {"dq": st["dq"], "dk": st["dk_"], "dv": st["dv_"], "dg": st["dg"], "dbeta": st["dbeta"],
                "dS0": st["dS0"]}
    if kind == "delta_step":
        T.ttt_delta_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], st["o"], st["batch"], st["dm"],
                         st["io"], slots=st["slot"], scale=st["scale"])
        return {"o": st["o"], "S": st["S"]}
    if kind == "norm_fwd":
        T.ttt_block_norm(st["y"], st["xo"], st["rows"], st["cfg"], X=st["x"], Z=st["z"], w_post=st["w_post"],
                         res_scale=st["lam"], w_pre=st["w_pre"], N=st["n"])
        return {"xo": st["xo"], "n": st["n"]}
    T.ttt_block_norm_backward(st["y"], st["dxo"], st["dy"], st["rows"], st["cfg"], st["ws"], X=st["x"], Z=st["z"],
                              w_post=st["w_post"], res_scale=st["lam"], w_pre=st["w_pre"], dN=st["dn"], dX=st["dx"],
                              dZ=st["dz"], dw_post=st["dw_post"], dres_scale=st["dlam"], dw_pre=st["dw_pre"])
    return {"dy": st["dy"], "dx": st["dx"], "dz": st["dz"], "dw_post": st["dw_post"], "dlam": st["dlam"],
            "dw_pre": st["dw_pre"]}


# --------------------------------------------------------------------------- the plain forms


def run(state):
    with torch.no_grad():
        if own:
            return _own(state)
        return {"delta_fwd": _plain_delta_fwd, "delta_bwd": _plain_delta_bwd, "delta_step": _plain_delta_step,
                "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[state["kind"]](state)


def _heads(t, h, rep=1):
    """[rows][h * d] -> fp32 [rows][h * rep][d], each head repeated for the value heads that share it."""
    t = t.float().reshape(t.shape[0], h, -1)
    return t.repeat_interleave(rep, 1) if rep > 1 else t


def _unit(t):
    return t / t.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)


def _pad_index(st):
    """Packed row of each token of [sequence][padded position], the chunk count, and which are tokens."""
    m = max(1, max(st["lens_list"]))
    nc = -(-m // CHUNK)
    pos = torch.arange(nc * CHUNK, device="cuda")
    cu = st["cu"].long()
    idx = cu[:-1, None] + pos[None]
    live = pos[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, idx, 0), live, nc


def _chunks(t, idx, live, nc):
    """[rows][heads][d] -> [sequence][head][chunk][position][d], zero behind each sequence."""
    x = t[idx] * live[..., None, None]
    N, L, H, d = x.shape
    return x.permute(0, 2, 1, 3).reshape(N, H, nc, CHUNK, d)


def _unchunk(x, live):
    """The inverse of _chunks: packed rows [rows][heads][d]."""
    N, H, nc, C, d = x.shape
    return x.reshape(N, H, nc * C, d).permute(0, 2, 1, 3)[live]


def _chunk_parts(st):
    rep = st["hv"] // st["hk"]
    idx, live, nc = _pad_index(st)
    q = _chunks(_unit(_heads(st["q"], st["hk"], rep)) * st["scale"], idx, live, nc)
    k = _chunks(_unit(_heads(st["k"], st["hk"], rep)), idx, live, nc)
    v = _chunks(_heads(st["v"], st["hv"]), idx, live, nc)
    # the decay's exponents reach far below zero inside a chunk: their sums and differences are in 64 bits
    c = _chunks(st["g"].double()[..., None], idx, live, nc).cumsum(-2)
    b = _chunks(st["beta"].float()[..., None], idx, live, nc)
    low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device="cuda").tril()
    D = torch.where(low, c - c.transpose(-1, -2), -math.inf).exp().float()
    L = (D * (k @ k.transpose(-1, -2))).tril(-1)
    P = D * (q @ k.transpose(-1, -2))
    # (I + beta L)^-1 for the strictly lower beta L: the product of I + (-beta L)^(2^i)
    X = -b * L
    eye = torch.eye(CHUNK, device="cuda")
    M = eye + X
    for _ in range(5):
        X = X @ X
        M = M + M @ X
    last = c[..., -1:, :]
    return idx, live, q, k, v, b, c.exp().float(), (last - c).exp().float(), last.exp().float(), L, P, M


def _start_state(st):
    return st["S0"].clone() if st["S0"] is not None else torch.zeros((st["N"], st["hv"], st["dv"], st["dk"]),
                                                                     device="cuda")


def _plain_delta_fwd(st):
    idx, live, q, k, v, b, ec, el, eG, L, P, M = _chunk_parts(st)
    S, out = _start_state(st), torch.empty_like(v)
    for i in range(q.shape[2]):
        R = v[:, :, i] - ec[:, :, i] * (k[:, :, i] @ S.transpose(-1, -2))
        U = M[:, :, i] @ (b[:, :, i] * R)
        out[:, :, i] = ec[:, :, i] * (q[:, :, i] @ S.transpose(-1, -2)) + P[:, :, i] @ U
        S = eG[:, :, i] * S + (el[:, :, i] * U).transpose(-1, -2) @ k[:, :, i]
    return {"o": _unchunk(out, live).reshape(st["T"], -1).to(st["v"].dtype), "S": S}


def _plain_delta_bwd(st):
    rep, hk = st["hv"] // st["hk"], st["hk"]
    idx, live, q, k, v, b, ec, el, eG, L, P, M = _chunk_parts(st)
    nc = q.shape[2]
    do = _chunks(_heads(st["do"], st["hv"]), idx, live, nc)
    S, states = _start_state(st), []
    E, U = torch.empty_like(v), torch.empty_like(v)
    for i in range(nc):
        states.append(S)
        R = v[:, :, i] - ec[:, :, i] * (k[:, :, i] @ S.transpose(-1, -2))
        U[:, :, i] = M[:, :, i] @ (b[:, :, i] * R)
        E[:, :, i] = R - L[:, :, i] @ U[:, :, i]
        S = eG[:, :, i] * S + (el[:, :, i] * U[:, :, i]).transpose(-1, -2) @ k[:, :, i]
    dS = st["dS"].clone() if st["dS"] is not None else torch.zeros_like(S)
    Z, dq, dk, dc = torch.empty_like(v), torch.empty_like(q), torch.empty_like(k), torch.empty_like(b)
    dlast = torch.empty_like(eG)
    for i in reversed(range(nc)):
        qi, ki, Ui, doi, ei, li = q[:, :, i], k[:, :, i], U[:, :, i], do[:, :, i], ec[:, :, i], el[:, :, i]
        dU = P[:, :, i].transpose(-1, -2) @ doi + li * (ki @ dS.transpose(-1, -2))
        Zi = M[:, :, i].transpose(-1, -2) @ dU
        Z[:, :, i] = Zi
        bz = b[:, :, i] * Zi
        low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device="cuda").tril()
        c = _decay(st, ec[:, :, i], low, i, idx, live, nc)
        F = c * (doi @ Ui.transpose(-1, -2))
        W = (c * (bz @ Ui.transpose(-1, -2))).tril(-1)
        dq_i = ei * (doi @ states[i]) + F @ ki
        read = -ei * (bz @ states[i]) - W @ ki
        hold = li * (Ui @ dS)
        write = F.transpose(-1, -2) @ qi - W.transpose(-1, -2) @ ki
        dq[:, :, i], dk[:, :, i] = dq_i, read + hold + write
        kept = (hold * ki).sum(-1, keepdim=True)
        flow = ((dq_i * qi).sum(-1, keepdim=True) + (read * ki).sum(-1, keepdim=True)
                - (write * ki).sum(-1, keepdim=True))
        after = flow.flip(-2).cumsum(-2).flip(-2)
        dlast[:, :, i] = eG[:, :, i] * (states[i] * dS).sum((-1, -2), keepdim=True)
        dc[:, :, i] = after + (kept.cumsum(-2) - kept) + dlast[:, :, i]
        dS = eG[:, :, i] * dS + (ei * doi).transpose(-1, -2) @ qi - (ei * bz).transpose(-1, -2) @ ki
    dt = st["q"].dtype

    def through_unit(t, grad, scale):
        x = _heads(t, hk)
        n = x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)
        grad = _unchunk(grad, live).reshape(st["T"], hk, rep, -1).sum(2) * scale
        u = x / n
        return ((grad - u * (u * grad).sum(-1, keepdim=True)) / n).reshape(st["T"], -1).to(dt)

    return {"dq": through_unit(st["q"], dq, st["scale"]), "dk": through_unit(st["k"], dk, 1.0),
            "dv": _unchunk(b * Z, live).reshape(st["T"], -1).to(dt), "dg": _unchunk(dc, live)[..., 0],
            "dbeta": _unchunk((E * Z).sum(-1, keepdim=True), live)[..., 0],
            "dS0": dS if st["s0"] else None}


def _decay(st, ec, low, i, idx, live, nc):
    """exp(c_i - c_j) on and below the diagonal of chunk i."""
    at = slice(i * CHUNK, (i + 1) * CHUNK)
    c = (st["g"].double()[idx[:, at]] * live[:, at, None]).cumsum(1).transpose(1, 2)[..., None]
    return torch.where(low, c - c.transpose(-1, -2), -math.inf).exp().float()


def _plain_delta_step(st):
    rep = st["hv"] // st["hk"]
    rows = st["slot"] >= 0
    at = torch.where(rows, st["slot"], 0).long()
    q = _unit(_heads(st["q"], st["hk"], rep)) * st["scale"]
    k = _unit(_heads(st["k"], st["hk"], rep))
    v = _heads(st["v"], st["hv"])
    S = st["S"][at] * st["g"].float().exp()[..., None, None]
    u = st["beta"].float()[..., None] * (v - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., None] * k[:, :, None, :]
    o = (S * q[:, :, None, :]).sum(-1).reshape(st["batch"], -1).to(st["o"].dtype)
    n = st["batch"] if st["batch"] <= 8 else st["batch"] - st["batch"] // 16  # the padding is at the end
    st["S"][at[:n]] = S[:n]
    st["o"][:n] = o[:n]
    return {"o": st["o"], "S": st["S"]}


def _f(t):
    return None if t is None else t.float()


def _norm_parts(st):
    y, G = st["y"].float(), st["group"]
    yg = y.reshape(y.shape[0], -1, G)
    ry = (yg.square().mean(-1, keepdim=True) + EPS).rsqrt()
    yh = (yg * ry).reshape(y.shape)
    w = st["w_post"].repeat(st["D"] // G)
    z = _f(st["z"])
    s = None if z is None else z / (1 + (-z).exp())
    p = yh * w if s is None else yh * w * s
    x = p if st["lam"] is None else st["lam"] * p
    x = x if st["x"] is None else st["x"].float() + x
    return ry, yh, w, z, s, p, x


def _plain_norm_fwd(st):
    ry, yh, w, z, s, p, x = _norm_parts(st)
    n = None if st["w_pre"] is None else x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["w_pre"]
    dt = st["y"].dtype
    return {"xo": x.to(dt), "n": None if n is None else n.to(dt)}


def _plain_norm_bwd(st):
    ry, yh, w, z, s, p, x = _norm_parts(st)
    dt, G = st["y"].dtype, st["group"]
    dx, dw_pre, dlam = st["dxo"].float(), None, None
    if st["dn"] is not None:
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        dn = st["dn"].float()
        a = dn * st["w_pre"]
        dx = dx + r * (a - x * r * r * (a * x).mean(-1, keepdim=True))
        dw_pre = (dn * x * r).sum(0)
    dp = dx
    if st["lam"] is not None:
        dlam = (dx * p).sum(0)
        dp = dx * st["lam"]
    t = dp if s is None else dp * s
    dw_post = (t * yh).reshape(t.shape[0], -1, G).sum((0, 1))
    dz = None
    if z is not None:
        sig = 1 / (1 + (-z).exp())
        dz = (dp * yh * w * sig * (1 + z * (1 - sig))).to(dt)
    dyh = (t * w).reshape(t.shape[0], -1, G)
    yg = yh.reshape(t.shape[0], -1, G)
    dy = (ry * (dyh - yg * (dyh * yg).mean(-1, keepdim=True))).reshape(t.shape)
    return {"dy": dy.to(dt), "dx": None if st["x"] is None else dx.to(dt), "dz": dz, "dw_post": dw_post, "dlam": dlam,
            "dw_pre": dw_pre}


# --------------------------------------------------------------------------- exact values


def exact(case, seed):
    """From the definitions, token by token, in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["kind"].startswith("norm"):
        return _exact_norm(st)
    with torch.no_grad():
        return _exact_step(st) if case["kind"] == "delta_step" else _exact_delta(st)


def _wide(t, heads, times):
    x = t.double().unflatten(1, (heads, t.shape[1] // heads))
    return torch.stack([x[:, h // times] for h in range(heads * times)], 1)


def _normed(x):
    return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True).clamp_min(1e-12)


def _exact_step(st):
    times = st["hv"] // st["hk"]
    q, k = _normed(_wide(st["q"], st["hk"], times)) * st["scale"], _normed(_wide(st["k"], st["hk"], times))
    v, S = _wide(st["v"], st["hv"], 1), st["S"].double().clone()
    o = torch.zeros_like(v)
    for b, s in enumerate(st["slot"].tolist()):
        if s < 0:
            continue
        decayed = S[s] * torch.exp(st["g"][b].double())[:, None, None]
        err = v[b] - torch.einsum("hij,hj->hi", decayed, k[b])
        S[s] = decayed + st["beta"][b].double()[:, None, None] * torch.einsum("hi,hj->hij", err, k[b])
        o[b] = torch.einsum("hij,hj->hi", S[s], q[b])
    return {"o": o.flatten(1), "S": S}


def _exact_delta(st):
    back, times = st["kind"] == "delta_bwd", st["hv"] // st["hk"]
    T, N, H, lens, dev = st["T"], st["N"], st["hv"], st["lens_list"], "cuda"
    if max(lens) * (4 if back else 1) > 200000:
        return None
    first = st["cu"][:-1].tolist()
    order = sorted(range(N), key=lambda i: -lens[i])  # the longest first: those still running are the first ones
    start = torch.tensor([first[i] for i in order], device=dev)
    q, k = _wide(st["q"], st["hk"], times), _wide(st["k"], st["hk"], times)
    qn, kn = q.norm(dim=-1, keepdim=True).clamp_min(1e-12), k.norm(dim=-1, keepdim=True).clamp_min(1e-12)
    q, k, v = q / qn, k / kn, _wide(st["v"], H, 1)
    alpha, beta, scale = st["g"].double().exp(), st["beta"].double(), st["scale"]
    S = torch.zeros((N, H, st["dv"], st["dk"]), dtype=torch.float64, device=dev)
    if st["S0"] is not None:
        S = st["S0"].double()[order].clone()
    counts = []
    n = N
    for t in range(max(lens) if lens else 0):
        while n and lens[order[n - 1]] <= t:
            n -= 1
        counts.append(n)

    def token(S, t):
        at = start[:counts[t]] + t
        kk, a, b = k[at][..., None], alpha[at][..., None, None], beta[at][..., None, None]
        held = a * S[:counts[t]]
        e = v[at][..., None] - held @ kk
        return at, kk, b, held, e, held + (b * e) * kk.mT

    if not back:
        o = torch.zeros((T, H, st["dv"]), dtype=torch.float64, device=dev)
        for t in range(len(counts)):
            at, kk, b, held, e, new = token(S, t)
            o[at] = (new @ q[at][..., None])[..., 0] * scale
            S[:counts[t]] = new
        out = torch.empty_like(S)
        out[order] = S
        return {"o": o.flatten(1), "S": out}

    every = 128
    kept = []
    for t in range(len(counts)):
        if t % every == 0:
            kept.append(S.clone())
        S[:counts[t]] = token(S, t)[-1]
    do = _wide(st["do"], H, 1)
    dS = torch.zeros_like(S) if st["dS"] is None else st["dS"].double()[order].clone()
    dq, dk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(alpha), torch.zeros_like(beta)
    for block in reversed(range(len(kept))):
        S, saved = kept[block], []
        for t in range(block * every, min(len(counts), (block + 1) * every)):
            at, kk, b, held, e, new = token(S, t)
            saved.append((at, kk, b, held, e, new))
            S = S.clone()
            S[:counts[t]] = new
        while saved:
            at, kk, b, held, e, new = saved.pop()
            n = len(at)
            d = do[at][..., None] * scale
            qq = q[at][..., None]
            G = dS[:n] + d * qq.mT
            dq[at] = (new.mT @ d)[..., 0]
            du = G @ kk
            db[at] = (du * e).sum((-1, -2))
            de = b * du
            dvv[at] = de[..., 0]
            G_held = G - de * kk.mT
            dk[at] = (G.mT @ (b * e) - held.mT @ de)[..., 0]
            dg[at] = (G_held * held).sum((-1, -2))
            dS[:n] = alpha[at][..., None, None] * G_held
    out = torch.empty_like(dS)
    out[order] = dS

    def raw(unit, norm, grad):
        grad = (grad - unit * (unit * grad).sum(-1, keepdim=True)) / norm
        return grad.unflatten(1, (st["hk"], times)).sum(2).flatten(1)

    return {"dq": raw(q, qn, dq), "dk": raw(k, kn, dk), "dv": dvv.flatten(1), "dg": dg, "dbeta": db,
            "dS0": out if st["s0"] else None}


def _exact_norm(st):
    """The definition in 64 bits, and its derivatives by differentiating that, in blocks of rows."""
    names = ("y", "x", "z", "w_post", "lam", "w_pre")
    weights = {n: st[n].double().requires_grad_() for n in names[3:] if st[n] is not None}
    back, out = st["kind"] == "norm_bwd", {}
    for at in torch.arange(st["rows"], device="cuda").split(8192):
        a = {n: st[n][at].double().requires_grad_(back) for n in names[:3] if st[n] is not None}
        y = a["y"].unflatten(1, (-1, st["group"]))
        p = y / torch.sqrt(torch.mean(y ** 2, -1, keepdim=True) + EPS) * weights["w_post"]
        p = p.flatten(1)
        if "z" in a:
            p = p * a["z"] * torch.sigmoid(a["z"])
        xo = p * weights["lam"] if "lam" in weights else p
        if "x" in a:
            xo = a["x"] + xo
        n = None
        if "w_pre" in weights:
            n = xo / torch.sqrt(torch.mean(xo ** 2, -1, keepdim=True) + EPS) * weights["w_pre"]
        if back:
            s = (xo * st["dxo"][at]).sum() + ((n * st["dn"][at]).sum() if st["dn"] is not None else 0)
            s.backward()
            got = {"d" + m: a[m].grad for m in a}
        else:
            got = {"xo": xo.detach()} | ({} if n is None else {"n": n.detach()})
        for m, t in got.items():
            out.setdefault(m, []).append(t)
    res = {m: torch.cat(t) for m, t in out.items()}
    if back:
        res.update({"d" + m: w.grad for m, w in weights.items()})
        return {m: res.get(m) for m in ("dy", "dx", "dz", "dw_post", "dlam", "dw_pre")}
    return {m: res.get(m) for m in ("xo", "n")}


# --------------------------------------------------------------------------- work


def work(case):
    """Bytes: every input once, every output once.  Flops: the recurrence's products, 2 flops each."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"].startswith("norm"):
        R, D = case["rows"], case["D"]
        res, gate = int(case["residual"]), int(case["gate"])
        if case["kind"] == "norm_fwd":
            return {"bytes": R * D * e * (2 + 2 * res + gate) + 4 * (case["group"] + 2 * res * D), "flops": 12 * R * D}
        return {"bytes": R * D * e * (3 + 3 * res + 2 * gate) + 8 * (case["group"] + 2 * res * D), "flops": 40 * R * D}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    per_token = e * (2 * hk * dk + 2 * hv * dv) + 8 * hv
    state = 4 * hv * dk * dv
    if case["kind"] == "delta_step":
        live = case["batch"] if case["batch"] <= 8 else case["batch"] - case["batch"] // 16
        return {"bytes": live * (per_token + 2 * state), "flops": live * hv * 6 * dk * dv}
    T, N = sum(_lens(case)), len(_lens(case))
    if case["kind"] == "delta_fwd":
        return {"bytes": T * per_token + N * state * (1 + int(case["s0"])), "flops": T * hv * 6 * dk * dv}
    return {"bytes": T * (e * (4 * hk * dk + 3 * hv * dv) + 16 * hv) + 3 * int(case["s0"]) * N * state,
            "flops": T * hv * 18 * dk * dv}
