"""What is measured of the selective state space operators and the verification of drafts.

A case names an operator ("op"), its sizes and its types.  `run` computes it in
a plain form (elementary torch operations in float32, or in 64 bits where
values lie next to a border) or, with `own` set, through the library's entry
points, on the same inputs.

  conv    the short causal convolution before a scan: a few taps a channel over
          ragged rows, the rows' last inputs in a slot-indexed pool
  scan    d = softplus(dt + bias); S <- exp(d A) S + d x B, y = C S + D x,
          out = y silu(z), a state of K values for every channel, for ragged rows
          over a slot-indexed pool
  accept  which drafted tokens the target's probabilities let through, from
          given random numbers, and the token drawn behind them

Prompts and single tokens move the pools on by whole rows.  Drafts ("drafts") are
first run without keeping a state, and the accepted part of each row is then
run once more into the pools.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # serving prompts: the rows of this repository's ragged prefill and the channels of its
        # projection (2 * 16 * 128 + 32 * 128)
        _conv("conv prompt ragged", rows=8, shortest=512, longest=4096, lens=2, pad=0, drafts=False, channels=8192,
              width=4, tokens="bf16", pool="f32", act="silu", bias=True),
        # this repository's decode batch: 256 rows, 8 of them padding
        _conv("conv step batch", rows=256, shortest=1, longest=1, lens=1, pad=8, drafts=False, channels=8192, width=4,
              tokens="bf16", pool="f32", act="silu", bias=True),
        # drafts of a speculative step in float32, an odd number of channels, three taps
        _conv("conv drafts odd", rows=64, shortest=2, longest=8, lens=4, pad=1, drafts=True, channels=2047, width=3,
              tokens="f32", pool="f32", act="none", bias=False),
        # serving prompts, the same rows, 32 heads of 128 channels with 16 states each
        _scan("scan prompt ragged", rows=8, shortest=512, longest=4096, lens=2, pad=0, drafts=False, nk=1, nv=32, K=16,
              V=128, tokens="bf16", dt="bf16", pool="f32", gate=True, skip=True),
        # one long document alone on the GPU: a long axis and half the channels
        _scan("scan one long", rows=1, shortest=16383, longest=16383, lens=1, pad=0, drafts=False, nk=1, nv=16, K=16,
              V=128, tokens="bf16", dt="bf16", pool="f32", gate=True, skip=True),
        # one user's decode step: latency
        _scan("scan step one row", rows=1, shortest=1, longest=1, lens=1, pad=0, drafts=False, nk=1, nv=32, K=16, V=128,
              tokens="bf16", dt="bf16", pool="f32", gate=True, skip=True),
        # the decode batch
        _scan("scan step batch", rows=256, shortest=1, longest=1, lens=1, pad=8, drafts=False, nk=1, nv=32, K=16, V=128,
              tokens="bf16", dt="bf16", pool="f32", gate=True, skip=True),
        # drafts of a speculative step, a bfloat16 pool, four groups of heads, step sizes in float32
        _scan("scan drafts", rows=64, shortest=2, longest=8, lens=4, pad=1, drafts=True, nk=4, nv=32, K=16, V=128,
              tokens="bf16", dt="f32", pool="bf16", gate=True, skip=True),
        # float32 activations, heads of odd width, more states than usual and no multiple of four, no gate
        _scan("scan odd f32", rows=5, shortest=3, longest=301, lens=6, pad=0, drafts=False, nk=3, nv=3, K=27, V=173,
              tokens="f32", dt="f32", pool="f32", gate=False, skip=False),
        # one user's drafts against a large vocabulary: latency
        _accept("accept one row", rows=1, shortest=9, longest=9, lens=1, vocab=131072, probs="f32", drafter=True),
        # a serving batch, four to seven drafts a row
        _accept("accept batch", rows=256, shortest=5, longest=8, lens=5, vocab=32000, probs="f32", drafter=True),
        # drafts without probabilities (looked up, not sampled), bfloat16 probabilities, an odd vocabulary
        _accept("accept looked up", rows=33, shortest=1, longest=6, lens=7, vocab=50257, probs="bf16", drafter=False),
    ]


def _conv(name=None, **c):
    return {**({"name": name} if name else {}), "op": "conv", **c}


def _scan(name=None, **c):
    return {**({"name": name} if name else {}), "op": "scan", **c}


def _accept(name=None, **c):
    return {**({"name": name} if name else {}), "op": "accept", **c}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


#: Work of the largest listed case, in bytes or operations / 50: a drawn one has no more.
MOST = 5.4e8


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if max(w["bytes"], w["flops"] / 50) > MOST:
            continue
        if c["op"] == "scan" and c["rows"] * c["longest"] * c["nv"] * c["V"] > 1 << 28:  # the plain form pads rows
            continue
        if c["op"] == "accept" and c["rows"] * c["longest"] * c["vocab"] > 1 << 27:
            continue
        return c


def _draw(rng):
    op = rng.choice(["conv", "scan", "scan", "accept"])
    if op == "accept":
        longest = rng.randint(2, 12)
        return _accept(rows=_log_int(rng, 1, 300), shortest=rng.randint(1, longest), longest=longest,
                       lens=rng.randrange(1000), vocab=_log_int(rng, 1000, 150000), probs=rng.choice(["f32", "f32", "bf16"]),
                       drafter=rng.random() < 0.7)
    kind = rng.choice(["prompt", "prompt", "step", "drafts"])
    if kind == "prompt":
        rows, longest = _log_int(rng, 1, 64), _log_int(rng, 9, 16384)
        lengths = {"rows": rows, "shortest": _log_int(rng, 1, longest), "longest": longest}
    elif kind == "step":
        lengths = {"rows": _log_int(rng, 1, 300), "shortest": 1, "longest": 1}
    else:
        longest = rng.randint(2, 8)
        lengths = {"rows": _log_int(rng, 1, 200), "shortest": rng.randint(1, longest), "longest": longest}
    lengths["lens"] = rng.randrange(1000)
    lengths["pad"] = rng.choice([0, 0, lengths["rows"] // 16])
    lengths["drafts"] = kind == "drafts"
    tokens = rng.choice(["bf16", "bf16", "f32"])
    pool = rng.choice(["f32", "f32", "bf16"])
    if op == "conv":
        channels = _log_int(rng, 100, 8192)
        channels = channels if rng.random() < 0.3 else max(64, channels // 64 * 64)
        return _conv(**lengths, channels=channels, width=rng.choice([2, 3, 4, 4]), tokens=tokens, pool=pool,
                     act=rng.choice(["silu", "silu", "none"]), bias=rng.random() < 0.7)
    nk = rng.choice([1, 1, 2, 4])
    V = _log_int(rng, 32, 512)
    V = V if rng.random() < 0.3 else max(32, V // 32 * 32)
    return _scan(**lengths, nk=nk, nv=nk * _log_int(rng, 1, max(1, 5000 // (nk * V))), K=rng.choice([8, 16, 16, 16, 27, 32, 64]),
                 V=V, tokens=tokens, dt=rng.choice([tokens, "f32"]), pool=pool, gate=rng.random() < 0.7,
                 skip=rng.random() < 0.7)


def _lengths(c):
    """Row lengths, by the case alone; the last `pad` rows are padding requests (slot -1) with tokens of their own."""
    r = random.Random(c["lens"])
    lens = [r.randint(c["shortest"], c["longest"]) for _ in range(c["rows"])]
    lens[0] = c["longest"]
    return lens


def _kept(c):
    """Tokens of each row that are accepted, where the case runs drafts."""
    r = random.Random(c["lens"] + 1)
    return [r.randint(1, n) for n in _lengths(c)]


def work(c):
    lens = _lengths(c)
    if c["op"] == "accept":
        # a target row for each row's draw; the drafter's beside it where a draft was refused: most rows of several
        refused = sum(1 - 0.6 ** (n - 1) for n in lens) if c["drafter"] else 0
        n = c["vocab"] * (len(lens) + refused)
        return {"bytes": n * SIZE[c["probs"]] + 16 * sum(lens) + 4 * len(lens) * (c["longest"] + 3), "flops": 2.0 * n}
    live = sum(lens[:c["rows"] - c["pad"]])
    rows = c["rows"] - c["pad"]
    if c["op"] == "conv":
        C, taps = c["channels"], c["width"] - 1
        return {"bytes": (live + sum(lens)) * C * SIZE[c["tokens"]] + 2 * rows * C * taps * SIZE[c["pool"]] +
                4 * C * (c["width"] + c["bias"]), "flops": live * C * (2.0 * c["width"] + (4 if c["act"] == "silu" else 0))}
    C, K = c["nv"] * c["V"], c["K"]
    token = C * (SIZE[c["tokens"]] * (1 + c["gate"]) + SIZE[c["dt"]]) + 2 * c["nk"] * K * SIZE[c["tokens"]]
    # a state's step: the decay's exponent and power, the input's product, two multiply-adds
    return {"bytes": live * token + sum(lens) * C * SIZE[c["tokens"]] + 2 * rows * C * K * SIZE[c["pool"]] +
            4 * C * (K + 1 + c["skip"]), "flops": live * C * (7.0 * K + 10)}


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, lens = case, _lengths(case)
    T, rows = sum(lens), c["rows"]

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": c, "T": T, "longest": c["longest"],
         "offsets": torch.tensor([sum(lens[:b]) for b in range(rows + 1)], dtype=torch.int32, device="cuda")}
    if c["op"] == "accept":
        # a peaked target, a drafter near it, and what the drafter drew
        logits = normal(T, c["vocab"], std=3.0)
        target = torch.softmax(logits, -1)
        draft = torch.softmax(logits.add_(normal(T, c["vocab"], std=0.7)), -1)
        del logits
        drawn = torch.empty(T, dtype=torch.int64, device="cuda")
        for t in range(0, T, 512):
            drawn[t:t + 512] = torch.multinomial(draft[t:t + 512], 1, generator=g)[:, 0]
        tokens = torch.randint(c["vocab"], (T,), generator=g, device="cuda")
        tokens[1:] = drawn[:-1]  # a row's first token is its last accepted one; whatever stands there is not looked at
        return {**s, "target": target.to(TYPES[c["probs"]]), "draft": draft.to(TYPES[c["probs"]]) if c["drafter"] else None,
                "tokens": tokens.to(torch.int32), "uniforms": uniform(T), "row_uniforms": uniform(rows)}
    slots = rows + max(2, rows // 2)
    slot = torch.randperm(slots - 1, generator=g, device="cuda")[:rows].to(torch.int32)  # the last slot is nobody's
    if c["pad"]:
        slot[rows - c["pad"]:] = -1
    s["slot"] = slot
    s["counts"] = torch.tensor(_kept(c), dtype=torch.int32, device="cuda") if c["drafts"] else None
    tok, pool = TYPES[c["tokens"]], TYPES[c["pool"]]
    if c["op"] == "conv":
        C = c["channels"]
        return {**s, "x": normal(T, C, dtype=tok), "weight": normal(C, c["width"], std=0.5),
                "bias": normal(C, std=0.1) if c["bias"] else None, "pool": normal(slots, C, c["width"] - 1).to(tok).to(pool)}
    nk, nv, K, V = c["nk"], c["nv"], c["K"], c["V"]
    # x has passed the convolution's SiLU; the gate is the second half of one input projection, B and C are
    # parts of one small projection
    x = normal(T, nv, V)
    x.copy_(x * torch.sigmoid(x))
    xz = normal(T, 2 * nv * V, dtype=tok) if c["gate"] else None
    bc = normal(T, 2 * nk * K, dtype=tok)
    # step sizes spread from 0.001 to 0.1 about their bias, rates from 1 to 16
    middle = torch.exp(math.log(1e-3) + math.log(1e2) * uniform(nv, V))
    rate = torch.exp(math.log(16.0) * uniform(nv, K, V))
    return {**s, "x": x.to(tok), "dt": normal(T, nv, V, std=0.5).to(TYPES[c["dt"]]),
            "dt_bias": torch.log(torch.expm1(middle)), "A": -rate, "B": bc[:, :nk * K].view(T, nk, K),
            "C": bc[:, nk * K:].view(T, nk, K), "z": xz[:, nv * V:].view(T, nv, V) if c["gate"] else None,
            "D": 1 + normal(nv, V, std=0.1) if c["skip"] else None, "pool": normal(slots, nv, K, V, std=0.5).to(pool)}


# ---- one pass -------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_conv(s):
    import gated_deltanet_linear_gdr_gb300 as gdr
    call = (s["x"], s["weight"], s["bias"], s["pool"], s["slot"], s["offsets"])
    act = "silu" if s["case"]["act"] == "silu" else None
    if s["counts"] is None:
        out = gdr.gdr_short_conv(*call, activation=act, max_row_len=s["longest"])
    else:
        out = gdr.gdr_short_conv(*call, activation=act, max_row_len=s["longest"], keep_state=False)
        gdr.gdr_short_conv(*call, activation=act, max_row_len=s["longest"], counts=s["counts"], state_only=True)
    return {"out": out, "state": s["pool"]}


def _own_scan(s):
    import gated_deltanet_linear_gdr_gb300 as gdr
    call = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], s["slot"], s["offsets"])
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "dt_softplus": True, "max_row_len": s["longest"]}
    if s["counts"] is None:
        out = gdr.gdr_selective_scan(*call, **more)
    else:
        out = gdr.gdr_selective_scan(*call, **more, keep_state=False)
        gdr.gdr_selective_scan(*call, **more, counts=s["counts"], state_only=True)
    return {"out": out, "state": s["pool"]}


def _own_accept(s):
    import gated_deltanet_linear_gdr_gb300 as gdr
    tokens, counts = gdr.gdr_accept_drafts(s["target"], s["draft"], s["tokens"], s["offsets"], s["uniforms"],
                                           s["row_uniforms"], max_row_len=s["longest"])
    return {"tokens": tokens, "counts": counts}


def _padded(s):
    """Every row's token indices, all rows as long as the longest, which of them exist, each token's row, its place there."""
    dev, offsets = s["offsets"].device, s["offsets"].long()
    start, length = offsets[:-1], offsets[1:] - offsets[:-1]
    at = torch.arange(s["longest"], device=dev)
    valid = at[None, :] < length[:, None]
    idx = torch.where(valid, start[:, None] + at[None, :], torch.zeros_like(at)[None, :])
    token = torch.arange(s["T"], device=dev)
    row = torch.searchsorted(offsets, token, right=True) - 1
    return idx, valid, row, token - start[row]


def _plain_conv(s):
    c = s["case"]
    taps, slot = c["width"] - 1, s["slot"].long()
    idx, valid, row, place = _padded(s)
    live = slot >= 0
    old = s["pool"][slot].float().transpose(1, 2)  # [rows, taps, channels], oldest first
    seen = torch.cat([old, torch.where(valid[..., None], s["x"][idx].float(), 0.0)], 1)
    y = torch.zeros_like(seen[:, taps:])
    if s["bias"] is not None:
        y = y + s["bias"]
    for m in range(c["width"]):
        y = y + s["weight"][:, m] * seen[:, m:m + s["longest"]]
    if c["act"] == "silu":
        y = y * torch.sigmoid(y)
    out = torch.where(live[row][:, None], y[row, place], 0.0).to(s["x"].dtype)
    kept = valid.sum(1) if s["counts"] is None else s["counts"].long()
    last = kept[:, None] + torch.arange(taps, device=kept.device)[None, :]
    new = torch.gather(seen, 1, last[..., None].expand(-1, -1, seen.shape[2])).transpose(1, 2)
    s["pool"][slot[live]] = new[live].to(s["pool"].dtype)
    return {"out": out, "state": s["pool"]}


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_scan(s):
    """Runs of tokens, all rows at once: powers and products of a run, then its states one after the other."""
    c = s["case"]
    r, slot = c["nv"] // c["nk"], s["slot"].long()
    idx, valid, row, place = _padded(s)
    live = slot >= 0
    d = torch.where(valid[..., None, None], _softplus(s["dt"].float() + s["dt_bias"])[idx], 0.0)
    x = s["x"].float()[idx] * d
    B, C = (s[n].float()[idx].repeat_interleave(r, 2) for n in ("B", "C"))
    state = s["pool"][slot].float()
    kept = valid.sum(1) if s["counts"] is None else s["counts"].long()
    keep = torch.zeros_like(state)
    y = torch.empty(d.shape, device=d.device)
    run = max(1, min(64, (1 << 27) // state.numel()))
    for t in range(0, s["longest"], run):
        dt = d[:, t:t + run, :, None, :]
        power = torch.exp(dt * s["A"]).unbind(1)
        states = B[:, t:t + run, :, :, None] * x[:, t:t + run, :, None, :]
        for i, now in enumerate(states.unbind(1)):
            state = now.addcmul_(power[i], state)
        y[:, t:t + run] = (states * C[:, t:t + run, :, :, None]).sum(3)
        at = kept - 1 - t  # the state to keep is a row's own at that place
        inside = (at >= 0) & (at < states.shape[1])
        mine = states[torch.arange(len(at), device=at.device), at.clamp(0, states.shape[1] - 1)]
        keep = torch.where(inside[:, None, None, None], mine, keep)
    y = y[row, place]
    if s["D"] is not None:
        y = y + s["D"] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    s["pool"][slot[live]] = keep[live].to(s["pool"].dtype)
    return {"out": torch.where(live[row][:, None, None], y, 0.0).to(s["x"].dtype), "state": s["pool"]}


def _plain_accept(s):
    """Comparisons and sums in 64 bits: a draft or a token next to a border must not fall to the other side."""
    start, width = s["offsets"][:-1].long(), s["longest"]
    drafts = s["offsets"][1:].long() - start - 1
    at = torch.arange(width - 1, device=start.device)
    there = at[None, :] < drafts[:, None]
    pos = torch.where(there, start[:, None] + at[None, :], torch.zeros_like(at)[None, :])
    token = s["tokens"].long()[(pos + 1).clamp(max=s["T"] - 1)]
    p = s["target"][pos, token].double()
    q = torch.ones_like(p) if s["draft"] is None else s["draft"][pos, token].double()
    passed = there & (s["uniforms"][pos].double() * q < p)
    count = torch.cumprod(passed.long(), 1).sum(1)
    final = start + count
    refused = count < drafts
    weight = s["target"][final].double()
    if s["draft"] is None:
        no = token.gather(1, count[:, None].clamp(max=max(width - 2, 0))) if width > 1 else torch.zeros_like(start)[:, None]
        other = torch.zeros_like(weight).scatter_(1, no, 1.0)
    else:
        other = s["draft"][final].double()
    weight = torch.where(refused[:, None], (weight - other).clamp(min=0), weight)
    total = weight.sum(1, keepdim=True)
    weight = torch.where(total > 0, weight, s["target"][final].double())
    upto = torch.cumsum(weight, 1)
    beyond = upto > s["row_uniforms"].double()[:, None] * upto[:, -1:]
    drawn = torch.where(beyond.any(1), beyond.int().argmax(1), (upto < upto[:, -1:]).sum(1))
    place = torch.arange(width, device=start.device)[None, :]
    out = torch.full((len(start), width), -1, dtype=torch.int64, device=start.device)
    out[:, :width - 1] = torch.where(place[:, :-1] < count[:, None], token, -1)
    out = torch.where(place == count[:, None], drawn[:, None], out)
    return {"tokens": out.to(torch.int32), "counts": (count + 1).to(torch.int32)}


_run_own = {"conv": _own_conv, "scan": _own_scan, "accept": _own_accept}
_run_plain = {"conv": _plain_conv, "scan": _plain_scan, "accept": _plain_accept}


# ---- in 64 bits, from the definitions -------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, lens = case, _lengths(case)
    off = [sum(lens[:b]) for b in range(c["rows"] + 1)]
    if c["op"] == "accept":
        return _exact_accept(s, off)
    slots = [int(x) for x in s["slot"].tolist()]
    live = [b for b in range(c["rows"]) if slots[b] >= 0]
    kept = _kept(c) if c["drafts"] else lens
    pool = s["pool"].double()
    if c["op"] == "conv":
        out = torch.zeros(s["T"], c["channels"], dtype=torch.float64, device="cuda")
        taps, w = c["width"] - 1, s["weight"].double()
        for b in live:
            seen = torch.cat([pool[slots[b]].T, s["x"][off[b]:off[b + 1]].double()])
            y = sum(seen[m:m + lens[b]] * w[:, m] for m in range(c["width"]))
            y = y if s["bias"] is None else y + s["bias"].double()
            out[off[b]:off[b + 1]] = y / (1 + torch.exp(-y)) if c["act"] == "silu" else y
            pool[slots[b]] = seen[kept[b]:kept[b] + taps].T
        return {"out": out, "state": pool}
    if s["longest"] * (1.2e-4 + c["rows"] * c["nv"] * c["K"] * c["V"] * 1e-10) > 20:
        return None
    # token by token: the t-th token of every row that has one, the longest rows first
    r, A = c["nv"] // c["nk"], s["A"].double()
    out = torch.zeros(s["T"], c["nv"], c["V"], dtype=torch.float64, device="cuda")
    order = sorted(live, key=lambda b: -lens[b])
    first = torch.tensor([off[b] for b in order], device="cuda", dtype=torch.long)
    state = pool[torch.tensor([slots[b] for b in order], device="cuda", dtype=torch.long)]
    active = len(order)
    ends = {}
    for i, b in enumerate(order):
        ends.setdefault(kept[b], []).append(i)
    for t in range(lens[order[0]] if order else 0):
        while lens[order[active - 1]] <= t:
            active -= 1
        tok = first[:active] + t
        v = s["dt"][tok].double() + s["dt_bias"].double()
        d = torch.logaddexp(v, torch.zeros_like(v))
        x = s["x"][tok].double()
        now = state[:active]
        now.mul_(torch.exp(d[:, :, None] * A)).addcmul_(s["B"][tok].double().repeat_interleave(r, 1)[..., None], (d * x)[:, :, None])
        y = torch.einsum("bhkv,bhk->bhv", now, s["C"][tok].double().repeat_interleave(r, 1))
        if s["D"] is not None:
            y = y + s["D"].double() * x
        if s["z"] is not None:
            z = s["z"][tok].double()
            y = y * z / (1 + torch.exp(-z))
        out[tok] = y
        for i in ends.get(t + 1, ()):
            pool[slots[order[i]]] = state[i]
    return {"out": out, "state": pool}


def _exact_accept(s, off):
    """Row by row, as the rule reads."""
    width = s["longest"]
    tokens = torch.full((len(off) - 1, width), -1, dtype=torch.int32)
    counts = torch.zeros(len(off) - 1, dtype=torch.int32)
    ids, u, v = s["tokens"].tolist(), s["uniforms"].tolist(), s["row_uniforms"].tolist()
    T = s["T"]
    nxt = torch.tensor(ids[1:] + [0], device="cuda")[:, None]
    p = s["target"].gather(1, nxt).double()[:, 0].tolist()
    q = [1.0] * T if s["draft"] is None else s["draft"].gather(1, nxt).double()[:, 0].tolist()
    for b in range(len(off) - 1):
        t, end = off[b], off[b + 1] - 1
        while t < end and u[t] * q[t] < p[t]:
            tokens[b, t - off[b]] = ids[t + 1]
            t += 1
        w = s["target"][t].double()
        if t < end:
            if s["draft"] is None:
                rest = w.clone()
                rest[ids[t + 1]] = 0
            else:
                rest = torch.relu(w - s["draft"][t].double())
            w = rest if bool((rest > 0).any()) else w
        upto = torch.cumsum(w, 0)
        x = int(torch.searchsorted(upto, v[b] * float(upto[-1]), right=True))
        tokens[b, t - off[b]] = x if x < len(w) else int(torch.nonzero(w)[-1])
        counts[b] = t - off[b] + 1
    return {"tokens": tokens.cuda(), "counts": counts.cuda()}
