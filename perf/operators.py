"""What the layer operators are measured on: the gated linear recurrence over long packed sequences with its backward
pass (``kda_scan``, ``kda_scan_backward``) and the per-head norm of queries and keys with the position rotation in the
same pass (``kda_qk_norm_rope``, ``kda_qk_norm_rope_backward``).

``own = False`` computes each operator with elementary torch operations in 32 bits (64 where 32 lose what matters);
``own = True`` makes the package's calls.  ``exact`` computes the definitions token by token in 64 bits.

The recurrence, per sequence and head, on the state S [K, V]:
    S' = Diag(exp(g_t)) S;  r_t = v_t - S'^T k_t;  S = S' + beta_t k_t r_t^T;  o_t = scale S^T q_t
The norm and rotation, per row and head: y = x rsqrt(sum x^2 + eps) ("l2") or x rsqrt(mean x^2 + eps) w ("rms"), then
each pair (a, b) of the first R components becomes m (a cos - b sin, a sin + b cos) at the angle position * frequency.
"""
import math

import torch

own = False

K = V = 128  # key and value width of a head, as in every configuration of this repository
CHUNK = 64   # tokens per chunk of the plain form


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One short prompt of a chat turn: latency of the launch chain counts.
        dict(name="scan_short", op="scan", lens="37", heads=8, decay="softplus", state=True),
        # A serving batch of prompts of different lengths, packed, each continuing its own state (8 local heads).
        dict(name="scan_packed", op="scan", lens="1024,1,777,2048,130,64,3001,1147", heads=8, decay="softplus", state=True),
        # One long document: the chain over its chunks is what bounds it.
        dict(name="scan_long", op="scan", lens="8192", heads=8, decay="mild", state=False),
        # A training step on a small ragged batch, with gradients from the final state.
        dict(name="train_small", op="train", lens="100,1,219", heads=4, decay="softplus", state=True),
        # A training step on one long sequence at 8 local heads.
        dict(name="train_long", op="train", lens="8192", heads=8, decay="mild", state=False),
        # A training step on packed documents with all 32 heads of a layer on one device: the throughput case.
        dict(name="train_packed", op="train", lens="1024,33,1999,1040", heads=32, decay="softplus", state=True),
        # A decode step's queries and keys: 32 sequences, 8 local heads, the unit norm of a linear-attention layer.
        dict(name="qk_decode", op="qk", rows=32, heads=8, kheads=8, dim=128, norm="l2", rot=0, inter=False, yarn=False),
        # A decode step with weights, half of each head rotated, far positions with scaled frequencies.
        dict(name="qk_decode_rope", op="qk", rows=256, heads=32, kheads=8, dim=128, norm="rms", rot=64, inter=False, yarn=True),
        # A packed prompt of a whole layer: bandwidth counts.
        dict(name="qk_prompt", op="qk", rows=16384, heads=32, kheads=32, dim=128, norm="l2", rot=128, inter=True, yarn=False),
        # Gradients of a small ragged batch, narrow heads, no norm (rotation alone).
        dict(name="qk_train_small", op="qk_train", rows=333, heads=4, kheads=2, dim=64, norm="none", rot=64, inter=False, yarn=False),
        # Gradients of a training batch with the weights' own gradients.
        dict(name="qk_train", op="qk_train", rows=16384, heads=32, kheads=8, dim=128, norm="rms", rot=128, inter=False, yarn=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "train", "qk", "qk_train"])
    if op in ("scan", "train"):
        heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
        tokens = _log_int(rng, 1, min(8192, 4096 * 32 // heads))
        n = min(tokens, rng.choice([1, 1, 2, 3, 5, 8, 16]))
        cuts = sorted(rng.sample(range(1, tokens), n - 1)) if n > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
        return dict(op=op, lens=",".join(map(str, lens)), heads=heads, decay=rng.choice(["softplus", "mild"]),
                    state=rng.random() < 0.5)
    dim = rng.choice([64, 96, 128, 256])
    rot = rng.choice([0, dim // 4 // 16 * 16, dim // 2, dim])
    norm = rng.choice(["l2", "rms"] if rot == 0 else ["none", "l2", "rms"])
    heads = rng.choice([1, 2, 4, 8, 16, 32])
    kheads = rng.choice([h for h in (1, 2, 4, 8, 16, 32) if h <= heads])
    rows = _log_int(rng, 1, 16384 * 128 // dim if heads + kheads > 32 else 16384)
    return dict(op=op, rows=rows, heads=heads, kheads=kheads, dim=dim, norm=norm, rot=rot,
                inter=rng.random() < 0.5, yarn=rng.random() < 0.5)


# --------------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _scan_inputs(case, seed):
    gen, H = _gen(seed), case["heads"]
    lens = [int(n) for n in case["lens"].split(",")]
    T = sum(lens)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    q, k, v = _unit(randn(T, H, K)).bfloat16(), _unit(randn(T, H, K)).bfloat16(), randn(T, H, V).bfloat16()
    if case["decay"] == "softplus":  # strong decays: a memory of a few tokens
        g = -torch.nn.functional.softplus(randn(T, H, K))
    else:  # a layer's decays as it is initialised: exp(g) mostly in (0.8, 1)
        rate = 1.0 + 15.0 * torch.rand(H, 1, generator=gen, device="cuda")
        dt = 0.001 + 0.099 * torch.rand(H, K, generator=gen, device="cuda")
        g = -rate * torch.nn.functional.softplus(randn(T, H, K) * 0.5 + torch.log(torch.expm1(dt)))
    beta = torch.sigmoid(randn(T, H))
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    st = dict(op=case["op"], lens=lens, q=q, k=k, v=v, g=g, beta=beta, cu=cu, scale=K ** -0.5, state=None)
    if case["state"]:
        st["state"] = randn(len(lens), H, K, V) * 0.02
    if case["op"] == "train":
        st["do"] = randn(T, H, V).bfloat16()
        st["dfinal"] = randn(len(lens), H, K, V) * 0.02 if case["state"] else None
    return st


def _frequencies(dim_rot, base, yarn):
    """Rotation frequencies in 64 bits and the factor on cos and sin: geometric, or with the low frequencies divided by
    16 for contexts 16 times the 4096 tokens trained on (a linear ramp between 32 and 1 turns per trained context)."""
    i = torch.arange(0, dim_rot, 2, dtype=torch.float64)
    f = base ** (-i / dim_rot)
    if not yarn:
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)

    def index(n):  # the (fractional) pair that makes n turns within the trained context
        return dim_rot * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), dim_rot - 1)
    ramp = ((torch.arange(turns.numel(), dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / 16.0 * ramp, 0.1 * math.log(16.0) + 1.0


def _qk_inputs(case, seed):
    gen, R, H, HK, D = _gen(seed), case["rows"], case["heads"], case["kheads"], case["dim"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    packed = randn(R, (H + 2 * HK) * D).bfloat16()  # one projection's rows: q, k and v side by side
    st = dict(op=case["op"], norm=case["norm"], inter=case["inter"], eps=1e-6, wq=None, wk=None, pos=None, freq=None, mscale=1.0)
    st["q"] = packed[:, :H * D].unflatten(-1, (H, D))
    st["k"] = packed[:, H * D:(H + HK) * D].unflatten(-1, (HK, D))
    if case["norm"] == "rms":
        st["wq"], st["wk"] = (1 + 0.1 * randn(D)).bfloat16(), (1 + 0.1 * randn(D)).bfloat16()
    if case["rot"]:
        freq, st["mscale"] = _frequencies(case["rot"], 10000.0, case["yarn"])
        st["freq"] = freq.cuda()
        if case["op"] == "qk" and case["rows"] <= 1024:  # decode rows: each sequence at its own far position
            st["pos"] = torch.randint(0, 1 << 20, (R,), generator=gen, device="cuda", dtype=torch.int32)
        else:  # packed sequences of 2048 tokens from a random start
            start = torch.randint(0, 1 << 17, (1,), generator=gen, device="cuda", dtype=torch.int32)
            st["pos"] = (torch.arange(R, device="cuda", dtype=torch.int32) % 2048 + start)
    if case["op"] == "qk_train":
        st["dq"], st["dk"] = randn(R, H, D).bfloat16(), randn(R, HK, D).bfloat16()
    return st


def prepare(case, seed):
    return (_scan_inputs if case["op"] in ("scan", "train") else _qk_inputs)(case, seed)


# ------------------------------------------------------------------------------------------------------------------ run
def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "scan":
        return _plain_scan(st, *(st[n] for n in ("q", "k", "v", "g", "beta")), st["state"])
    if st["op"] == "train":
        return _plain_train(st)
    return _plain_qk(st) if st["op"] == "qk" else _plain_qk_train(st)


def _run_own(st):
    import linear_attention_recurrent_decode_b200 as kda
    if st["op"] == "scan":
        out, final = kda.kda_scan(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], cu_seqlens=st["cu"], scale=st["scale"])
        return {"out": out, "final": final}
    if st["op"] == "train":
        if "ws" not in st:  # a training program keeps one workspace per layer
            n, (T, H) = len(st["lens"]), st["beta"].shape
            st["ws"] = torch.empty(kda.scan_workspace_bytes(T, n, H, training=True), dtype=torch.uint8, device="cuda")
        a = (st["q"], st["k"], st["v"], st["g"], st["beta"])
        out, final = kda.kda_scan(*a, st["state"], cu_seqlens=st["cu"], scale=st["scale"], workspace=st["ws"], save=True)
        dq, dk, dv, dg, dbeta, ds = kda.kda_scan_backward(st["do"], *a, st["state"], d_final_state=st["dfinal"], cu_seqlens=st["cu"],
                                                          scale=st["scale"], workspace=st["ws"], saved=True)
        return {"out": out, "final": final, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dstate": ds}
    kw = dict(norm=st["norm"], eps=st["eps"], q_weight=st["wq"], k_weight=st["wk"], positions=st["pos"], inv_freq=st["freq"],
              interleaved=st["inter"], rope_scale=st["mscale"])
    if st["op"] == "qk":
        q, k = kda.kda_qk_norm_rope(st["q"], st["k"], **kw)
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = kda.kda_qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], **kw)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ---- the plain scan: chunks of 64 tokens, batched products within them, a loop over the chunks of the longest sequence
def _pad_index(st, device):
    """Index of each padded (sequence, chunk, token) slot into the packed tokens, T for the padding."""
    lens, T = st["lens"], st["q"].shape[0]
    nc = max(1, max((n + CHUNK - 1) // CHUNK for n in lens))
    t = torch.arange(nc * CHUNK, device=device)
    n, start = st["cu"][1:] - st["cu"][:-1], st["cu"][:-1]
    return torch.where(t < n[:, None], start[:, None] + t, T).long().view(len(lens), nc, CHUNK)


def _pad(x, idx):
    """[T, H, ...] -> [N, C, H, 64, ...] in 32 bits, zeros in the padding."""
    x = torch.cat([x.float(), x.new_zeros(1, *x.shape[1:]).float()])[idx]
    return x.movedim(3, 2)


def _plain_core(st, q, k, v, g, beta, S):
    """Outputs [N, C, H, 64, V] and final states from padded inputs; differentiable."""
    N, C, H = q.shape[:3]
    gam = g.double().cumsum(-2)  # cumulative log-decay from the chunk's start
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    A, P = [], []
    for h in range(H):  # head by head: the pairwise decays of all heads at once would not leave room
        gh = gam[:, :, h]
        E = torch.exp((gh.unsqueeze(-2) - gh.unsqueeze(-3)).masked_fill(~tri.unsqueeze(-1), -math.inf).float())
        Ek = E * k[:, :, h].unsqueeze(-3)  # [.., t, s, i]
        A.append((Ek @ k[:, :, h].unsqueeze(-1)).squeeze(-1).tril(-1))
        P.append((Ek @ q[:, :, h].unsqueeze(-1)).squeeze(-1))
    A, P = torch.stack(A, 2), torch.stack(P, 2)
    b = beta.unsqueeze(-1)
    M = -b * A  # (I + beta A)^-1 = prod (I + M^(2^j)): M is nilpotent
    inv = torch.eye(CHUNK, device=q.device) + M
    for _ in range(5):
        M = M @ M
        inv = inv + inv @ M
    e = torch.exp(gam.float())
    end = gam[..., -1:, :]
    W, U0 = inv @ (b * k * e), inv @ (b * v)
    kend, qe, dec = k * torch.exp((end - gam).float()), q * e, torch.exp(end.float()).squeeze(-2).unsqueeze(-1)
    outs = []
    for c in range(C):
        U = U0[:, c] - W[:, c] @ S
        outs.append(qe[:, c] @ S + P[:, c] @ U)
        S = dec[:, c] * S + kend[:, c].transpose(-1, -2) @ U
    return st["scale"] * torch.stack(outs, 1), S


def _zero_state(st):
    return torch.zeros(len(st["lens"]), st["q"].shape[1], K, V, device=st["q"].device)


def _plain_scan(st, q, k, v, g, beta, S):
    idx = _pad_index(st, q.device)
    o, S = _plain_core(st, *(_pad(x, idx) for x in (q, k, v, g, beta)), _zero_state(st) if S is None else S)
    out = o.new_empty(q.shape[0] + 1, *v.shape[1:])
    out[idx] = o.movedim(2, 3)
    return {"out": out[:-1].bfloat16(), "final": S}


def _plain_train(st):
    idx, T = _pad_index(st, st["q"].device), st["q"].shape[0]
    leaves = [_pad(st[n], idx).requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    S0 = (_zero_state(st) if st["state"] is None else st["state"].clone()).requires_grad_()
    with torch.enable_grad():
        o, S = _plain_core(st, *leaves, S0)
    do = _pad(st["do"], idx)
    grads = torch.autograd.grad([o, S], leaves + [S0], [do, torch.zeros_like(S) if st["dfinal"] is None else st["dfinal"]])

    def unpad(x, like):
        y = x.new_empty(T + 1, *like.shape[1:])
        y[idx] = x.detach().movedim(2, 3)
        return y[:-1].to(like.dtype)

    got = {"out": unpad(o, st["v"]), "final": S.detach()}
    for n, gr in zip(("q", "k", "v", "g", "beta"), grads):
        got["d" + n] = unpad(gr, st[n])
    got["dstate"] = grads[-1]
    return got


# ---- the plain norm and rotation
def _angles(st):
    """cos and sin [rows, 1, R/2], the angles in 64 bits."""
    a = st["pos"].double()[:, None, None] * st["freq"]
    return (torch.cos(a) * st["mscale"]).float(), (torch.sin(a) * st["mscale"]).float()


def _rotate(x, cos, sin, inter):
    r = 2 * cos.shape[-1]
    if inter:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), x[..., r:]], -1)
    a, b = x[..., :r // 2], x[..., r // 2:r]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., r:]], -1)


def _inverse_norm(st, x):
    s = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((s / x.shape[-1] if st["norm"] == "rms" else s) + st["eps"])


def _plain_qk(st):
    got = {}
    for n, w in (("q", "wq"), ("k", "wk")):
        x = st[n].float()
        if st["norm"] != "none":
            x = x * _inverse_norm(st, x)
        if st[w] is not None:
            x = x * st[w].float()
        if st["freq"] is not None:
            x = _rotate(x, *_angles(st), st["inter"])
        got[n] = x.bfloat16()
    return got


def _plain_qk_train(st):
    got, dws = {}, {}
    for n, w in (("q", "wq"), ("k", "wk")):
        x, dy = st[n].float(), st["d" + n].float()
        if st["freq"] is not None:  # the rotation's transpose turns back
            cos, sin = _angles(st)
            dy = _rotate(dy, cos, -sin, st["inter"])
        dws["dw" + n] = None
        if st["norm"] != "none":
            inv = _inverse_norm(st, x)
            xh = x * inv
            if st[w] is not None:
                dws["dw" + n] = (dy * xh).double().sum((0, 1)).float()
                dy = dy * st[w].float()
            m = (dy * xh).sum(-1, keepdim=True)
            dy = inv * (dy - xh * (m / x.shape[-1] if st["norm"] == "rms" else m))
        got["d" + n] = dy.bfloat16()
    return {**got, **dws}


# ----------------------------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] in ("scan", "train"):
        lens, H = [int(n) for n in case["lens"].split(",")], case["heads"]
        th, states = sum(lens) * H, len(lens) * H * K * V * 4
        ins, out = th * (2 * K * 2 + V * 2 + K * 4 + 4), th * V * 2
        # per token and head: decay (K V), then S^T k, the rank-1 write and S^T q at 2 K V each
        if case["op"] == "scan":
            return {"bytes": ins + out + states * (1 + case["state"]), "flops": 7 * K * V * th}
        # forward, then q do^T, dS^T k, dS r, S' dr, k dr^T, S . dS, S do at 2 K V each and the decay; the gradients written
        # are as large as the inputs read
        return {"bytes": ins * 2 + out * 2 + states * (2 + 2 * case["state"]), "flops": 22 * K * V * th}
    n = case["rows"] * (case["heads"] + case["kheads"]) * case["dim"]
    return {"bytes": n * 2 * (2 if case["op"] == "qk" else 3) + case["rows"] * 4, "flops": n * (8 if case["op"] == "qk" else 16)}


# ---------------------------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_scan(st) if case["op"] in ("scan", "train") else _exact_qk(st)


def _exact_scan(st):
    """The definition token by token in 64 bits, every sequence of the batch at once; then its adjoint, backwards."""
    lens, (T, H) = st["lens"], st["beta"].shape
    if max(lens) * len(lens) * H > 300_000 or (st["op"] == "train" and max(lens) * len(lens) * H * K * V * 8 > 60e9):
        return None
    N, L, dev = len(lens), max(lens), st["q"].device
    idx = torch.full((L, N), T, device=dev)
    for n, ln in enumerate(lens):
        idx[:ln, n] = torch.arange(ln, device=dev) + int(st["cu"][n])
    q, k, v, g, beta = (torch.cat([st[x].double(), st[x].new_zeros(1, *st[x].shape[1:]).double()])[idx] for x in ("q", "k", "v", "g", "beta"))
    S = (_zero_state(st) if st["state"] is None else st["state"]).double()
    train = st["op"] == "train"
    before = torch.empty(L, N, H, K, V, dtype=torch.float64, device=dev) if train else None  # states ahead of each token
    out, rs = torch.zeros(T + 1, H, V, dtype=torch.float64, device=dev), []
    for t in range(L):
        if train:
            before[t] = S
        Sd = torch.exp(g[t])[..., None] * S
        r = v[t] - (k[t][..., None] * Sd).sum(-2)
        S = Sd + (beta[t][..., None] * k[t])[..., None] * r[..., None, :]
        out[idx[t]] = st["scale"] * (q[t][..., None] * S).sum(-2)
        rs.append(r)
    got = {"out": out[:-1], "final": S}
    if not train:
        return got
    do = torch.cat([st["do"].double(), st["do"].new_zeros(1, H, V).double()])[idx] * st["scale"]
    dS = torch.zeros_like(S) if st["dfinal"] is None else st["dfinal"].double()
    res = {n: torch.zeros(T + 1, *st[n].shape[1:], dtype=torch.float64, device=dev) for n in ("q", "k", "v", "g", "beta")}
    for t in reversed(range(L)):
        Sd = torch.exp(g[t])[..., None] * before[t]
        bk, r = beta[t][..., None] * k[t], rs[t]
        St = Sd + bk[..., None] * r[..., None, :]
        res["q"][idx[t]] = (St * do[t][..., None, :]).sum(-1)
        dS = dS + q[t][..., None] * do[t][..., None, :]
        dkr = (dS * r[..., None, :]).sum(-1)                 # the gradient of beta k
        dr = (dS * bk[..., None]).sum(-2)
        res["beta"][idx[t]] = (dkr * k[t]).sum(-1)
        res["v"][idx[t]] = dr
        res["k"][idx[t]] = beta[t][..., None] * dkr - (Sd * dr[..., None, :]).sum(-1)
        dSd = dS - k[t][..., None] * dr[..., None, :]
        res["g"][idx[t]] = (dSd * Sd).sum(-1)
        dS = torch.exp(g[t])[..., None] * dSd
    got.update({"d" + n: x[:-1] for n, x in res.items()})
    got["dstate"] = dS
    return got


def _exact_qk(st):
    """In 64 bits, the rotation as a complex product and the gradients by differentiating the definition."""
    got, dws = {}, {}
    for n, w in (("q", "wq"), ("k", "wk")):
        x = st[n].double().requires_grad_()
        wt = None if st[w] is None else st[w].double().requires_grad_()
        with torch.enable_grad():
            y = x
            if st["norm"] == "l2":
                y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) + st["eps"])
            elif st["norm"] == "rms":
                y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + st["eps"])
            if wt is not None:
                y = y * wt
            if st["freq"] is not None:
                r = 2 * st["freq"].numel()
                turn = torch.polar(torch.full((), st["mscale"], dtype=torch.float64, device=x.device), st["pos"].double()[:, None, None] * st["freq"])
                if st["inter"]:
                    z = turn * torch.view_as_complex(y[..., :r].unflatten(-1, (-1, 2)).contiguous())
                    y = torch.cat([torch.view_as_real(z).flatten(-2), y[..., r:]], -1)
                else:
                    z = turn * torch.complex(y[..., :r // 2], y[..., r // 2:r])
                    y = torch.cat([z.real, z.imag, y[..., r:]], -1)
        if st["op"] == "qk":
            got[n] = y.detach()
        else:
            gr = torch.autograd.grad(y, [x] + ([] if wt is None else [wt]), st["d" + n].double())
            got["d" + n], dws["dw" + n] = gr[0], gr[1] if len(gr) > 1 else None
    return {**got, **dws}
