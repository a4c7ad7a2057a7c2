"""What is measured of the layer operators: decayed linear attention and the fused block norms.

A case names an operator ("op"), its sizes and its types.  `run` computes it
in a plain form (elementary torch operations in float32, rounded once) or,
with `own` set, through the library's entry points, on the same inputs.

  linattn    S <- lambda_h S + k v^T, o = scale S^T q, for ragged rows over a
             slot-indexed state pool updated in place (prompts, drafts, single
             tokens)
  gate_norm  per-head norm of a recurrence's output times its activated gate
  residual_norm  h' = h + a act(g) N(block), y = N(h'): a block's output norm,
             gate, residual scale and add, and the next block's norm
"""
import math
import random

import torch

own = False

EPS = 1e-6
CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # serving prompts, the sizes of this repository's ragged prefill (nk=16, nv=32, K=V=128)
        _linattn("prompt ragged", rows=8, shortest=512, longest=4096, lens=2, pad=0, nk=16, nv=32, K=128, V=128,
                 tokens="bf16", pool="f32", log=True),
        # one long document alone on the GPU: few (row, head) pairs, a long axis
        _linattn("prompt one long", rows=1, shortest=16383, longest=16383, lens=1, pad=0, nk=32, nv=32, K=128, V=128,
                 tokens="bf16", pool="bf16", log=False),
        # a batch of chat turns, small heads, some requests padded
        _linattn("prompt chat turns", rows=48, shortest=9, longest=700, lens=3, pad=2, nk=16, nv=16, K=64, V=64,
                 tokens="bf16", pool="bf16", log=True),
        # drafts of a speculative step, values twice as wide as keys
        _linattn("drafts", rows=64, shortest=2, longest=8, lens=4, pad=1, nk=16, nv=16, K=128, V=256,
                 tokens="bf16", pool="bf16", log=True),
        # one user's decode step: latency
        _linattn("step one row", rows=1, shortest=1, longest=1, lens=1, pad=0, nk=16, nv=32, K=128, V=128,
                 tokens="bf16", pool="bf16", log=False),
        # this repository's decode batch: 256 rows, 8 of them padding
        _linattn("step batch", rows=256, shortest=1, longest=1, lens=1, pad=8, nk=16, nv=32, K=128, V=128,
                 tokens="bf16", pool="bf16", log=True),
        # a float32 pool behind float32 activations, odd batch and head counts
        _linattn("step f32", rows=93, shortest=1, longest=1, lens=1, pad=0, nk=3, nv=9, K=64, V=128,
                 tokens="f32", pool="f32", log=False),
        # the recurrence's float32 output on its way to the output projection, one decode batch
        _gate("gate norm step", tokens=256, heads=32, dim=128, x="f32", g="bf16", y="bf16", act="silu", first=False,
              centered=False, weight=True),
        # a prompt's heads
        _gate("gate norm prompt", tokens=15843, heads=32, dim=128, x="bf16", g="bf16", y="bf16", act="silu",
              first=False, centered=False, weight=True),
        # block boundary of a decode batch: pre-norm of the next block only after the add
        _residual("residual norm step", tokens=33, dim=4096, x="bf16", h="f32", y="bf16", post=False, gate="none",
                  act="none", centered=False),
        # block boundary of a prompt: norms on both sides, a gate per element
        _residual("residual norm prompt", tokens=8192, dim=4096, x="bf16", h="bf16", y="bf16", post=True,
                  gate="element", act="sigmoid", centered=False),
        # an odd width (rows not 16-byte aligned), centred norms, a float32 residual stream, a gate per channel
        _residual("residual norm odd", tokens=2111, dim=2047, x="bf16", h="f32", y="bf16", post=True, gate="channel",
                  act="none", centered=True),
    ]


def _linattn(name=None, **c):
    return {**({"name": name} if name else {}), "op": "linattn", **c}


def _gate(name=None, **c):
    return {**({"name": name} if name else {}), "op": "gate_norm", **c}


def _residual(name=None, **c):
    return {**({"name": name} if name else {}), "op": "residual_norm", **c}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


#: Work of the largest listed case, in bytes or operations / 50: a drawn one has no more.
MOST = 7.0e8


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        widths = [c.get("dim"), c.get("dim", 0) * c.get("heads", 0), c.get("tokens"), c.get("nv", 0) * c.get("V", 0),
                  c.get("nk", 0) * c.get("K", 0), c.get("longest")]
        if max(w["bytes"], w["flops"] / 50) <= MOST and 3 << 10 not in widths:
            return c


def _draw(rng):
    op = rng.choice(["prompt", "prompt", "step", "gate_norm", "residual_norm"])
    if op in ("prompt", "step"):
        heads = {"nk": _log_int(rng, 1, 32)}
        heads["nv"] = heads["nk"] * rng.choice([1, 1, 2, 3])
        pool = rng.choice(["bf16", "f32"])
        log = rng.random() < 0.5
    if op == "prompt":
        longest = _log_int(rng, 2, 16384)
        rows = _log_int(rng, 1, 64)
        return _linattn(rows=rows, shortest=_log_int(rng, 1, longest), longest=longest, lens=rng.randrange(1000),
                        pad=rng.choice([0, 0, 1]) if rows > 1 else 0, **heads, K=rng.choice([64, 128]),
                        V=rng.choice([64, 128, 128, 256]), tokens="bf16", pool=pool, log=log)
    if op == "step":
        rows = _log_int(rng, 1, 300)
        return _linattn(rows=rows, shortest=1, longest=1, lens=1, pad=rng.choice([0, 0, rows // 16]), **heads,
                        K=rng.choice([64, 128]), V=rng.choice([64, 128, 256]), tokens=rng.choice(["bf16", "f32"]),
                        pool=pool, log=log)
    if op == "gate_norm":
        return _gate(tokens=_log_int(rng, 1, 20000), heads=_log_int(rng, 1, 48),
                     dim=rng.choice([64, 80, 96, 128, 128, 160, 256]), x=rng.choice(["bf16", "f32"]),
                     g=rng.choice(["bf16", "f32"]), y="bf16", act=rng.choice(["silu", "sigmoid"]),
                     first=rng.random() < 0.3, centered=rng.random() < 0.3, weight=rng.random() < 0.8)
    gate = rng.choice(["none", "element", "token", "channel"])
    dim = _log_int(rng, 256, 8192)
    dim = dim if rng.random() < 0.4 else max(256, dim // 64 * 64)
    return _residual(tokens=_log_int(rng, 1, 16000), dim=dim, x=rng.choice(["bf16", "f32"]),
                     h=rng.choice(["bf16", "f32"]), y="bf16", post=rng.random() < 0.6, gate=gate,
                     act="none" if gate == "none" else rng.choice(["none", "sigmoid", "silu"]),
                     centered=rng.random() < 0.3)


def _lengths(c):
    """Row lengths, by the case alone; the last `pad` rows are padding requests (slot -1) with tokens of their own."""
    r = random.Random(c["lens"])
    lens = [r.randint(c["shortest"], c["longest"]) for _ in range(c["rows"])]
    lens[0] = c["longest"]
    return lens


def work(c):
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "linattn":
        lens = _lengths(c)
        live = lens[:c["rows"] - c["pad"]]
        t, nk, nv, K, V = sum(live), c["nk"], c["nv"], c["K"], c["V"]
        return {"bytes": t * (2 * nk * K + nv * V) * size[c["tokens"]] + sum(lens) * nv * V * size[c["tokens"]] +
                2 * len(live) * nv * K * V * size[c["pool"]] + 4 * nv, "flops": 4.0 * t * nv * K * V}
    if c["op"] == "gate_norm":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": n * (size[c["x"]] + size[c["g"]] + size[c["y"]]) + 4 * c["dim"], "flops": 10.0 * n}
    n = c["tokens"] * c["dim"]
    gate = {"none": 0, "element": n, "token": c["tokens"], "channel": c["dim"]}[c["gate"]] * size[c["x"]]
    return {"bytes": n * (size[c["x"]] + 2 * size[c["h"]] + size[c["y"]]) + gate + 8 * c["dim"], "flops": 12.0 * n}


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    c = case
    if c["op"] == "linattn":
        lens = _lengths(c)
        T, rows, nk, nv, K, V = sum(lens), c["rows"], c["nk"], c["nv"], c["K"], c["V"]
        # one packed projection [Q | K | V] a token; q and k have passed a SiLU feature map
        qkv = normal(T, 2 * nk * K + nv * V)
        qk = qkv[:, :2 * nk * K]
        qk.copy_(qk * torch.sigmoid(qk))
        qkv = qkv.to(TYPES[c["tokens"]])
        # decays of several scales: half-lives from under one token to hundreds
        slope = torch.exp2(-8.0 * torch.arange(1, nv + 1, device="cuda", dtype=torch.float32) / nv)
        slope = slope * (0.75 + 0.5 * torch.rand(nv, generator=g, device="cuda"))
        slots = rows + max(2, rows // 2)
        slot = torch.randperm(slots - 1, generator=g, device="cuda")[:rows].to(torch.int32)  # the last slot is nobody's
        if c["pad"]:
            slot[rows - c["pad"]:] = -1
        offsets = torch.tensor([sum(lens[:b]) for b in range(rows + 1)], dtype=torch.int32, device="cuda")
        return {"case": c, "T": T, "q": qkv[:, :nk * K].view(T, nk, K), "k": qkv[:, nk * K:2 * nk * K].view(T, nk, K),
                "v": qkv[:, 2 * nk * K:].view(T, nv, V), "decay": -slope if c["log"] else torch.exp(-slope),
                "pool": normal(slots, nv, K, V, dtype=TYPES[c["pool"]], std=0.5), "slot": slot, "offsets": offsets,
                "longest": c["longest"]}
    if c["op"] == "gate_norm":
        shape = (c["tokens"], c["heads"], c["dim"])
        return {"case": c, "x": normal(*shape, dtype=TYPES[c["x"]], std=2.0), "gate": normal(*shape, dtype=TYPES[c["g"]]),
                "weight": 1 + normal(c["dim"], std=0.1) if c["weight"] else None}
    T, D = c["tokens"], c["dim"]
    shape = {"none": None, "element": (T, D), "token": (T, 1), "channel": (D,)}[c["gate"]]
    return {"case": c, "block": normal(T, D, dtype=TYPES[c["x"]]), "residual": normal(T, D, dtype=TYPES[c["h"]], std=3.0),
            "gate": None if shape is None else normal(*shape, dtype=TYPES[c["x"]]), "weight": 1 + normal(D, std=0.1),
            "post": 1 + normal(D, std=0.1) if c["post"] else None, "scale": 0.7}


# ---- one pass -------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_linattn(s):
    import gated_deltanet_linear_gdr_gb300 as gdr
    out = gdr.gdr_linattn_fwd(s["q"], s["k"], s["v"], s["decay"], s["pool"], s["slot"], s["offsets"],
                              decay_is_log=s["case"]["log"], max_row_len=s["longest"])
    return {"out": out, "state": s["pool"]}


def _own_gate_norm(s):
    import gated_deltanet_linear_gdr_gb300 as gdr
    c = s["case"]
    return {"out": gdr.gdr_gate_norm(s["x"], s["gate"], s["weight"], eps=EPS, activation=c["act"], gate_first=c["first"],
                                     centered=c["centered"], out_dtype=TYPES[c["y"]])}


def _own_residual_norm(s):
    import gated_deltanet_linear_gdr_gb300 as gdr
    c = s["case"]
    h, y = gdr.gdr_residual_norm(s["block"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                                 activation=None if c["act"] == "none" else c["act"], residual_scale=s["scale"], eps=EPS,
                                 centered=c["centered"], out_dtype=TYPES[c["y"]])
    return {"residual": h, "out": y}


def _powers(decay, log, n):
    """lambda^n for whole n (float32); 0^0 = 1."""
    if log:
        return torch.where(n == 0, torch.ones_like(n), torch.exp(decay * n))
    return torch.pow(decay, n)


def _plain_step(s):
    """One token a row (longest == 1)."""
    c, live = s["case"], (s["slot"] >= 0)[:, None, None, None]
    r, tok, slot = c["nv"] // c["nk"], s["offsets"][:-1].long(), s["slot"].long()
    q, k = (s[n][tok].float().repeat_interleave(r, 1) for n in ("q", "k"))
    v, old = s["v"][tok].float(), s["pool"][slot]
    lam = (torch.exp(s["decay"]) if c["log"] else s["decay"])[None, :, None, None]
    state = lam * old.float() + k[..., :, None] * v[..., None, :]
    out = c["K"] ** -0.5 * (q[..., None] * state).sum(2)
    s["pool"][slot] = torch.where(live, state.to(old.dtype), old)
    return {"out": torch.where(live[..., 0], out, torch.zeros_like(out)).to(s["v"].dtype), "state": s["pool"]}


def _plain_linattn(s):
    """Chunks of CHUNK tokens, all rows padded to the longest, every chunk at once."""
    if s["longest"] == 1:
        return _plain_step(s)
    c, dev, C = s["case"], s["q"].device, CHUNK
    B, nk, nv, K, V, log = c["rows"], c["nk"], c["nv"], c["K"], c["V"], c["log"]
    N = -(-s["longest"] // C)
    start, slot = s["offsets"][:-1].long(), s["slot"].long()
    length = s["offsets"][1:].long() - start
    at = torch.arange(N * C, device=dev)
    valid = at[None, :] < length[:, None]
    idx = torch.where(valid, start[:, None] + at[None, :], torch.zeros_like(at)[None, :])

    def chunks(x, heads, dim):  # [T, heads, dim] -> [B, nv, N, C, dim] float32, zero past each row's end
        x = torch.where(valid[..., None, None], x[idx].float(), 0.0)
        return x.view(B, N, C, heads, dim).permute(0, 3, 1, 2, 4).repeat_interleave(nv // heads, 1)

    q, k, v = chunks(s["q"], nk, K), chunks(s["k"], nk, K), chunks(s["v"], nv, V)
    i = torch.arange(C, device=dev, dtype=torch.float32)
    lam = s["decay"]
    # within a chunk
    gap = i[:, None] - i[None, :]
    inside = torch.where(gap >= 0, _powers(lam[:, None, None], log, gap.clamp(min=0)), 0.0)  # [nv, C, C]
    out = ((q @ k.transpose(-1, -2)) * inside[None, :, None]) @ v
    # each chunk's own contribution to the state at its end
    n = (length[:, None] - torch.arange(N, device=dev)[None, :] * C).clamp(0, C).float()  # tokens in the chunk
    left = n[:, :, None] - 1 - i
    keep = torch.where(left[:, None] >= 0, _powers(lam[None, :, None, None], log, left[:, None].clamp(min=0)), 0.0)
    own_state = (k * keep[..., None]).transpose(-1, -2) @ v  # [B, nv, N, K, V]
    # the states at the chunks' starts, and the last one
    edge = torch.minimum(torch.arange(N + 1, device=dev)[None, :] * C, length[:, None]).float()  # [B, N + 1]
    far = edge[:, :, None] - edge[:, None, 1:]  # tokens from the end of chunk d to the start of chunk c
    before = torch.arange(N + 1, device=dev)[:, None] > torch.arange(N, device=dev)[None, :]
    carry = torch.where(before[None, None], _powers(lam[None, :, None, None], log, far[:, None].clamp(min=0)), 0.0)
    old = s["pool"][slot]
    states = (carry @ own_state.reshape(B, nv, N, K * V)).view(B, nv, N + 1, K, V)
    states = states + _powers(lam[None, :, None], log, edge[:, None])[..., None, None] * old.float()[:, :, None]
    out = out + _powers(lam[:, None], log, i + 1)[None, :, None, :, None] * (q @ states[:, :, :N])
    # back to tokens
    token = torch.arange(s["T"], device=dev)
    row = torch.searchsorted(s["offsets"].long(), token, right=True) - 1
    out = out.view(B, nv, N * C, V).transpose(1, 2)[row, token - start[row]] * K ** -0.5
    live = slot >= 0
    s["pool"][slot] = torch.where(live[:, None, None, None], states[:, :, N].to(old.dtype), old)
    return {"out": torch.where(live[row][:, None, None], out, 0.0).to(s["v"].dtype), "state": s["pool"]}


def _act(x, name):
    if name == "none":
        return x
    return x * torch.sigmoid(x) if name == "silu" else torch.sigmoid(x)


def _norm(x, weight, centered):
    if centered:
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x if weight is None else x * weight


def _plain_gate_norm(s):
    c = s["case"]
    x, g = s["x"].float(), _act(s["gate"].float(), c["act"])
    y = _norm(x * g, s["weight"], c["centered"]) if c["first"] else _norm(x, s["weight"], c["centered"]) * g
    return {"out": y.to(TYPES[c["y"]])}


def _plain_residual_norm(s):
    c = s["case"]
    u = s["block"].float()
    if s["post"] is not None:
        u = _norm(u, s["post"], c["centered"])
    if s["gate"] is not None:
        u = u * _act(s["gate"].float(), c["act"])
    h = s["residual"].float() + s["scale"] * u
    return {"residual": h.to(s["residual"].dtype), "out": _norm(h, s["weight"], c["centered"]).to(TYPES[c["y"]])}


_run_own = {"linattn": _own_linattn, "gate_norm": _own_gate_norm, "residual_norm": _own_residual_norm}
_run_plain = {"linattn": _plain_linattn, "gate_norm": _plain_gate_norm, "residual_norm": _plain_residual_norm}


# ---- in 64 bits, from the definitions -------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "linattn":
        if c["longest"] * (6e-5 + c["rows"] * c["nv"] * c["K"] * c["V"] * 1.5e-11) > 20:
            return None
        # token by token: every row's state advanced by its t-th token
        nv, r = c["nv"], c["nv"] // c["nk"]
        lam = s["decay"].double()
        lam = torch.exp(lam) if c["log"] else lam
        off = [int(x) for x in s["offsets"].tolist()]
        slots = [int(x) for x in s["slot"].tolist()]
        live = [b for b in range(c["rows"]) if slots[b] >= 0]
        pool = s["pool"].double()
        out = torch.zeros(s["T"], nv, c["V"], dtype=torch.float64, device="cuda")
        order = sorted(live, key=lambda b: off[b] - off[b + 1])  # longest first: the active rows are a prefix
        lens = [off[b + 1] - off[b] for b in order]
        first = torch.tensor([off[b] for b in order], device="cuda", dtype=torch.long)
        at = torch.tensor([slots[b] for b in order], device="cuda", dtype=torch.long)
        state = pool[at]
        active = len(order)
        for t in range(lens[0] if lens else 0):
            while lens[active - 1] <= t:
                active -= 1
            tok = first[:active] + t
            k = s["k"][tok].double().repeat_interleave(r, dim=1)
            q = s["q"][tok].double().repeat_interleave(r, dim=1)
            now = state[:active]
            now.mul_(lam[None, :, None, None]).addcmul_(k[..., None], s["v"][tok].double()[:, :, None, :])
            out[tok] = (now * q[..., None]).sum(dim=2) / math.sqrt(c["K"])
        pool[at] = state
        return {"out": out, "state": pool}

    def norm(x, w):
        if c["centered"]:
            x = x - x.sum(-1, keepdim=True) / x.shape[-1]
        x = x * torch.rsqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        return x if w is None else x * w.double()

    def act(x):
        return {"none": lambda: torch.ones_like(x) * x, "silu": lambda: x / (1 + torch.exp(-x)),
                "sigmoid": lambda: 1 / (1 + torch.exp(-x))}[c["act"]]()

    if c["op"] == "gate_norm":
        x, g = s["x"].double(), act(s["gate"].double())
        return {"out": norm(x * g, s["weight"]) if c["first"] else norm(x, s["weight"]) * g}
    u = s["block"].double()
    if s["post"] is not None:
        u = norm(u, s["post"])
    if s["gate"] is not None:
        u = act(s["gate"].double()) * u
    h = s["residual"].double() + s["scale"] * u
    return {"residual": h, "out": norm(h, s["weight"])}
