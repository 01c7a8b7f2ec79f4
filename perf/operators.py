"""Cases of the gated delta rule (whole prompts, single tokens) and of the gated norm behind it.

`run` computes an operator in plain torch, or, with `own` set, through this package's entry points.
The recurrence, per state head with the fp32 state S [K][V]:

    S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,    y_t = S_t^T q_t
"""
import math
import random

import torch

own = False

K = 128
EPS_QK = 1e-6
CHUNK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a short prompt of one user: latency
        dict(name="chunk_short", op="chunk", seqs=1, tokens=48, heads=32, qk_heads=32, vdim=128, dtype="bf16", normalize=True),
        # a server's prefill batch, q and k shared by two state heads, lengths all over the place
        dict(name="chunk_ragged", op="chunk", seqs=16, tokens=8192, heads=32, qk_heads=16, vdim=128, dtype="bf16", normalize=True),
        # one long document
        dict(name="chunk_long", op="chunk", seqs=1, tokens=8192, heads=32, qk_heads=32, vdim=128, dtype="bf16", normalize=False),
        # a large prefill batch
        dict(name="chunk_batch", op="chunk", seqs=48, tokens=32768, heads=32, qk_heads=32, vdim=128, dtype="bf16", normalize=True),
        # a shard of a layer with odd sizes, fp16
        dict(name="chunk_odd", op="chunk", seqs=7, tokens=2501, heads=12, qk_heads=4, vdim=80, dtype="f16", normalize=True),
        # the framework's own fp32 tensors
        dict(name="chunk_f32", op="chunk", seqs=24, tokens=1500, heads=32, qk_heads=32, vdim=128, dtype="f32", normalize=False),
        # one user's next token
        dict(name="step_one", op="step", rows=1, slots=64, heads=32, qk_heads=16, vdim=128, dtype="bf16", normalize=True),
        # a decode batch of the size of the GDN configuration
        dict(name="step_batch", op="step", rows=512, slots=512, heads=32, qk_heads=32, vdim=128, dtype="bf16", normalize=True),
        # a partly filled pool, fp32 tensors, odd sizes
        dict(name="step_odd", op="step", rows=61, slots=100, heads=12, qk_heads=4, vdim=80, dtype="f32", normalize=False),
        # the norm behind a small decode batch
        dict(name="norm_decode", op="norm", rows=16, groups=32, width=128, xdtype="bf16", dtype="bf16", act="silu", gate_first=False, shared=True),
        # the norm behind a prefill batch
        dict(name="norm_prompt", op="norm", rows=32768, groups=32, width=128, xdtype="bf16", dtype="bf16", act="silu", gate_first=False, shared=True),
        # the Mamba-2 layer of 128 heads of 80: 8 groups, the gate before the norm, behind the fp32 sketch decode
        dict(name="norm_grouped", op="norm", rows=256, groups=8, width=1280, xdtype="f32", dtype="bf16", act="silu", gate_first=True, shared=False),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "step", "norm"))
    if op == "norm":
        width = rng.choice((_log_int(rng, 2, 128) * 8, 64, 80, 128, 256))
        groups = _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, max(1, min(32768, 32768 * 32 * 128 // (2 * groups * width))))
        return dict(op=op, rows=rows, groups=groups, width=width, xdtype=rng.choice(("f32", "bf16", "bf16", "f16")),
                    dtype=rng.choice(("f32", "bf16", "bf16", "f16")), act=rng.choice(("silu", "silu", "sigmoid")),
                    gate_first=rng.random() < 0.4, shared=rng.random() < 0.6)
    qk = rng.choice((1, 2, 4, 5, 8, 16))
    heads = qk * rng.choice([r for r in (1, 2, 3, 4) if r * qk <= 32])
    c = dict(op=op, heads=heads, qk_heads=qk, vdim=rng.choice((16, 64, 80, 96, 128, 128, 128, 144, 256)),
             dtype=rng.choice(("bf16", "bf16", "bf16", "f16", "f32")), normalize=rng.random() < 0.6)
    room = 32 * 128 / (heads * c["vdim"])
    if op == "step":
        rows = _log_int(rng, 1, min(700, max(1, int(500 * room))))
        return dict(c, rows=rows, slots=rows + rng.randrange(0, 5))
    tokens = _log_int(rng, 1, int(min(16384 if c["dtype"] != "f32" else 2048, 30000 * room)))
    return dict(c, tokens=tokens, seqs=_log_int(rng, 1, min(40, tokens)))


def lengths(case):
    """The prompts' lengths: a ragged cut of the tokens that the case alone decides; some are empty."""
    r = random.Random(case["seqs"] * 1000003 + case["tokens"])
    cuts = sorted(r.randint(0, case["tokens"]) for _ in range(case["seqs"] - 1))
    ends = [0] + cuts + [case["tokens"]]
    return [b - a for a, b in zip(ends, ends[1:])]


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["groups"] * case["width"]
        w = 4 * case["width"] * (1 if case["shared"] else case["groups"])
        return {"bytes": n * (SIZES[case["xdtype"]] + 2 * SIZES[case["dtype"]]) + w, "flops": 10 * n}
    h, q, v, es = case["heads"], case["qk_heads"], case["vdim"], SIZES[case["dtype"]]
    if case["op"] == "step":
        n, states = case["rows"], case["rows"]
    else:
        n, states = case["tokens"], sum(length > 0 for length in lengths(case))
    return {"bytes": n * (2 * q * K + 2 * h * v) * es + n * h * 8 + states * (2 * h * K * v * 4 + 8), "flops": 6 * n * h * K * v}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        shape = (case["rows"], case["groups"], case["width"])
        x = randn(*shape).mul_(0.3).to(DTYPES[case["xdtype"]])
        z = randn(*shape).to(DTYPES[case["dtype"]])
        w = 1 + 0.1 * randn(*((shape[2],) if case["shared"] else shape[1:]))
        return dict(case=case, x=x, z=z, w=w, out=torch.empty(shape, dtype=z.dtype, device="cuda"))
    dt, h, hq, v = DTYPES[case["dtype"]], case["heads"], case["qk_heads"], case["vdim"]
    n = case["rows"] if case["op"] == "step" else case["tokens"]
    slots = case["slots"] if case["op"] == "step" else case["seqs"]
    q, k = randn(n, hq, K), randn(n, hq, K)
    if not case["normalize"]:  # the model has brought them to unit length itself
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    state = dict(
        case=case, q=q.to(dt), k=k.to(dt), v=randn(n, h, v).to(dt),
        a=torch.exp(-0.05 * torch.nn.functional.softplus(randn(n, h))),
        beta=torch.sigmoid(randn(n, h)),
        S=randn(slots, h, K, v).mul_(0.1),
        y=torch.empty(n, h, v, dtype=dt, device="cuda"),
        slot=torch.randperm(slots, generator=g, device="cuda").to(torch.int32),
        scale=K ** -0.5)
    if case["op"] == "step":
        state["slot"] = state["slot"][:n].contiguous()
    else:
        state["lens"] = lengths(case)
        ends = torch.tensor([0] + state["lens"]).cumsum(0)
        state["cu"] = ends.to(device="cuda", dtype=torch.int32)
        # the plain form pads the prompts to whole chunks: where each padded token lies, -1 for none
        longest = -(-max(state["lens"]) // CHUNK) * CHUNK
        at = torch.arange(longest)[None] + ends[:-1, None]
        state["at"] = torch.where(at < ends[1:, None], at, -1).cuda()
    if own:
        import rank_state_read_b200 as rs

        state["plan"] = rs.Plan("gdn", batch=slots, heads=h, qk_heads=hq, key_dim=K, value_dim=v, window=16, groups=1,
                                basis_rows=64, rank_cap=64, rank=[rs.DENSE] * h)
    return state


def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import rank_state_read_b200 as rs

    c = s["case"]
    if c["op"] == "norm":
        rs.sketchssm_gated_norm(s["x"], s["z"], s["w"], s["out"], eps=1e-6, activation=c["act"], gate_first=c["gate_first"])
        return {"out": s["out"]}
    how = dict(slot=s["slot"], normalize_qk=c["normalize"], scale=s["scale"])
    if c["op"] == "step":
        rs.sketchssm_delta_step(s["plan"], s["q"], s["k"], s["v"], s["a"], s["beta"], s["S"], s["y"], **how)
    else:
        rs.sketchssm_delta_chunk(s["plan"], s["cu"], s["q"], s["k"], s["v"], s["a"], s["beta"], s["S"], s["y"], **how)
    return {"y": s["y"], "S": s["S"]}


def _plain(s):
    return {"norm": _plain_norm, "step": _plain_step, "chunk": _plain_chunk}[s["case"]["op"]](s)


def _plain_norm(s):
    c = s["case"]
    x, z = s["x"].float(), s["z"].float()
    gate = torch.sigmoid(z)
    if c["act"] == "silu":
        gate = gate * z
    if c["gate_first"]:
        x = x * gate
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["w"]
    if not c["gate_first"]:
        x = x * gate
    s["out"].copy_(x)
    return {"out": s["out"]}


def _heads(s):
    """q, k of every state head and v in fp32, q scaled."""
    c = s["case"]
    q, k = s["q"].float(), s["k"].float()
    if c["normalize"]:
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + EPS_QK)
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + EPS_QK)
    r = c["heads"] // c["qk_heads"]
    return (q * s["scale"]).repeat_interleave(r, 1), k.repeat_interleave(r, 1), s["v"].float()


def _plain_step(s):
    q, k, v = _heads(s)
    slot = s["slot"].long()
    S = s["S"][slot] * s["a"][..., None, None]
    u = s["beta"][..., None] * (v - torch.einsum("bhkv,bhk->bhv", S, k))
    S = S + k[..., None] * u[..., None, :]
    s["y"].copy_(torch.einsum("bhkv,bhk->bhv", S, q))
    s["S"][slot] = S
    return {"y": s["y"], "S": s["S"]}


def _plain_chunk(s):
    q, k, v = _heads(s)
    at = s["at"]
    there = at >= 0
    idx = at.clamp(min=0)

    def padded(x):  # [seqs][heads][chunks][CHUNK][..], zeros past a prompt's end
        x = torch.where(there.view(there.shape + (1,) * (x.dim() - 1)), x[idx], x.new_zeros(()))
        x = x.transpose(1, 2)
        return x.reshape(x.shape[:2] + (-1, CHUNK) + x.shape[3:])

    slot = s["slot"].long()
    S = s["S"][slot]
    q, k, v, beta = padded(q), padded(k), padded(v), padded(s["beta"])
    G = padded(s["a"].double().log()).cumsum(-1)  # differences of these are what counts: 64 bits
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, (G[..., :, None] - G[..., None, :]).clamp(max=0).exp().float(), 0)
    first, last = G.exp().float(), (G[..., -1:] - G).exp().float()
    A = beta[..., None] * decay * (k @ k.transpose(-1, -2))
    P = decay * (q @ k.transpose(-1, -2))
    eye = torch.eye(CHUNK, device=q.device)
    T = torch.linalg.solve_triangular(A.tril(-1) + eye, eye.expand_as(A), upper=False, unitriangular=True)
    TV, TK = T @ (beta[..., None] * v), T @ ((beta * first)[..., None] * k)
    y = torch.empty_like(v)
    for c in range(q.shape[2]):  # the state goes from chunk to chunk
        U = TV[:, :, c] - TK[:, :, c] @ S
        y[:, :, c] = first[:, :, c, :, None] * (q[:, :, c] @ S) + P[:, :, c] @ U
        S = first[:, :, c, -1, None, None] * S + (last[:, :, c, :, None] * k[:, :, c]).transpose(-1, -2) @ U
    y = y.reshape(y.shape[:2] + (-1, y.shape[-1])).transpose(1, 2)
    s["y"].copy_(y[there])
    s["S"][slot] = S
    return {"y": s["y"], "S": s["S"]}


def exact(case, seed):
    """The definition, token by token in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, z, w = s["x"].double(), s["z"].double(), s["w"].double()
        act = z / (1 + torch.exp(-z)) if case["act"] == "silu" else 1 / (1 + torch.exp(-z))
        u = x * act if case["gate_first"] else x
        u = u / (u.square().sum(-1, keepdim=True) / case["width"] + 1e-6).sqrt() * w
        return {"out": u if case["gate_first"] else u * act}
    step = case["op"] == "step"
    starts = list(range(case["rows"])) if step else s["cu"][:-1].tolist()
    lens = [1] * case["rows"] if step else s["lens"]
    slot, S, y = s["slot"].tolist(), s["S"].double(), torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    of = torch.tensor([slot[i] for i in order], device="cuda")
    start = torch.tensor([starts[i] for i in order], device="cuda")
    head = torch.arange(case["heads"], device="cuda") // (case["heads"] // case["qk_heads"])
    M = S[of]
    for t in range(max(lens)):
        n = sum(length > t for length in lens)
        i = start[:n] + t
        q, k, v = s["q"][i].double()[:, head], s["k"][i].double()[:, head], s["v"][i].double()
        if case["normalize"]:
            q = q / (q.square().sum(-1, keepdim=True) + EPS_QK).sqrt()
            k = k / (k.square().sum(-1, keepdim=True) + EPS_QK).sqrt()
        a, beta = s["a"][i].double()[..., None, None], s["beta"][i].double()[..., None, None]
        m = M[:n]
        erased = (k[..., None, :] @ m)
        m -= beta * k[..., None] * erased
        m *= a
        m += beta * k[..., None] * v[..., None, :]
        y[i] = s["scale"] * (q[..., None, :] @ m)[..., 0, :]
    S[of] = M
    return {"y": y, "S": S}
