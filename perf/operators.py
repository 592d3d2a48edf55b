"""Dense attention beside the block-sparse kernels: what is measured of it.

Three operators, all bf16 with grouped heads (Hq query heads over Hkv key/value heads):

* "prompt": softmax attention over packed sequences of different lengths, causal (a row of query
  r of a sequence sees keys 0 .. r + kv_len - q_len) or full, with its log-sum-exp;
* "train": the gradients dq, dk, dv of the same;
* "decode": the newest tokens of many requests over a prefix they share, kept once, and over the
  keys of their own that follow it.

Cases hold plain values; lengths of packed sequences are texts such as "77,1,2048" ("q/kv" where
the two differ).
"""
import math

import torch

own = False

# the largest padded score matrices (elements, heads included) a drawn case may have in plain form
_MOST_SCORES = {"prompt": 40 * 15488 * 15488, "train": 40 * 8192 * 8192, "decode": 64 * 40 * 24576}


def listed():
    return [
        # one short prompt of a small head size: latency of a single call
        {"name": "prompt_short", "op": "prompt", "hq": 8, "hkv": 2, "d": 64, "lens": "77", "causal": True, "token_major": True},
        # a serving step's batch of prompts, some one token long, one resumed behind cached keys
        {"name": "prompts_ragged", "op": "prompt", "hq": 40, "hkv": 8, "d": 128, "lens": "1,641,130,2048,77,1,1000,512/1500,300", "causal": True, "token_major": True},
        # the four video clips of the packed block-sparse workload, attended in full (no mask)
        {"name": "clips_full", "op": "prompt", "hq": 12, "hkv": 12, "d": 128, "lens": "3000,6144/7040,9216", "causal": False, "token_major": False},
        # one long prompt, as long as the flagship video sequence
        {"name": "prompt_long", "op": "prompt", "hq": 40, "hkv": 8, "d": 128, "lens": "15488", "causal": True, "token_major": True},
        # gradients of a small packed batch with plain heads
        {"name": "train_small", "op": "train", "hq": 12, "hkv": 12, "d": 64, "lens": "77,641,300", "causal": True, "token_major": False},
        # a training step's pack of documents, seven query heads to a key head
        {"name": "train_packed", "op": "train", "hq": 56, "hkv": 8, "d": 128, "lens": "1025,2048,300,1500,777,1,2541", "causal": True, "token_major": True},
        # one long training sequence
        {"name": "train_long", "op": "train", "hq": 40, "hkv": 8, "d": 128, "lens": "8192", "causal": True, "token_major": True},
        # two requests behind a short system prompt: latency
        {"name": "decode_few", "op": "decode", "hq": 8, "hkv": 2, "d": 128, "batch": 2, "tokens": 1, "prefix": 500, "suffix": 100},
        # a few drafted tokens per request to be checked at once
        {"name": "decode_drafts", "op": "decode", "hq": 40, "hkv": 8, "d": 128, "batch": 16, "tokens": 5, "prefix": 4100, "suffix": 1000},
        # many answers sampled from one long prompt
        {"name": "decode_many", "op": "decode", "hq": 40, "hkv": 8, "d": 128, "batch": 64, "tokens": 1, "prefix": 15488, "suffix": 2048},
        # no common prefix: every request reads keys of its own only
        {"name": "decode_apart", "op": "decode", "hq": 56, "hkv": 8, "d": 128, "batch": 24, "tokens": 1, "prefix": 0, "suffix": 9216},
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _pairs_of(text):
    """[(q_len, kv_len)] of a case's lengths."""
    return [tuple(int(x) for x in (part.split("/") * 2)[:2]) for part in text.split(",")]


def _visible(q_len, kv_len, causal):
    """How many (query, key) pairs of one sequence take part."""
    if not causal:
        return q_len * kv_len
    first = kv_len - q_len + 1  # keys that row 0 sees
    skipped = max(0, 1 - first)  # rows that see none
    rows = q_len - skipped
    return rows * (max(first, 1) + kv_len) // 2 if rows > 0 else 0


def draw(rng):
    op = rng.choice(["prompt", "train", "decode"])
    while True:
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 4, 8, 12])
        hq = hkv * rng.choice([1, 2, 3, 5, 7, 8])
        case = {"op": op, "hq": hq, "hkv": hkv, "d": d}
        if op == "decode":
            case |= {"batch": _log_uniform(rng, 1, 64), "tokens": rng.choice([1, 1, 1, 2, 3, 5, 8]),
                     "prefix": rng.choice([0, 1]) * _log_uniform(rng, 1, 20000) if rng.random() < 0.4 else _log_uniform(rng, 1, 20000),
                     "suffix": _log_uniform(rng, 8, 12000)}
            if case["hq"] > 56 or case["batch"] * case["hq"] * case["tokens"] * (case["prefix"] + case["suffix"]) > _MOST_SCORES[op]:
                continue
            cost, most = work(case)["bytes"], work(listed()[9])["bytes"]
        else:
            longest = 15488 if op == "prompt" else 8192
            parts = []
            for _ in range(rng.choice([1, 1, 2, 3, 5, 9])):
                n = _log_uniform(rng, 1, longest)
                parts.append(str(n) if rng.random() < 0.7 else "%d/%d" % (n, min(longest, n + _log_uniform(rng, 1, 2000))))
            case |= {"lens": ",".join(parts), "causal": rng.random() < 0.8, "token_major": rng.random() < 0.5}
            pairs = _pairs_of(case["lens"])
            padded = len(pairs) * max(a for a, _ in pairs) * max(b for _, b in pairs) * hq
            if case["hq"] > 56 or padded > _MOST_SCORES[op] or sum(b for _, b in pairs) * hkv > 8 * 40000:
                continue
            cost, most = work(case)["flops"], work(listed()[3 if op == "prompt" else 6])["flops"]
        if cost <= most:
            return case


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    state = {"case": case, "scale": d ** -0.5}
    if case["op"] == "decode":
        b, t, s, p = case["batch"], case["tokens"], case["suffix"], case["prefix"]
        # token-major caches, as the projections write them, seen as [.., heads, keys, d]
        state["q"] = _normal((b, t, hq, d), gen).transpose(1, 2)
        state["k_prefix"] = _normal((p, hkv, d), gen).transpose(0, 1)
        state["v_prefix"] = _normal((p, hkv, d), gen).transpose(0, 1)
        state["k_suffix"] = _normal((b, s, hkv, d), gen).transpose(1, 2)
        state["v_suffix"] = _normal((b, s, hkv, d), gen).transpose(1, 2)
        # requests are at different points of their answers; the new tokens' keys are in the cache already
        share = torch.rand(b, generator=gen, device="cuda", dtype=torch.float64)
        state["lens"] = (t + (share * (s - t + 1)).floor().clamp_(0, s - t)).to(torch.int32)
        return state
    pairs = _pairs_of(case["lens"])
    cu_q, cu_kv = [0], [0]
    for a, b in pairs:
        cu_q.append(cu_q[-1] + a)
        cu_kv.append(cu_kv[-1] + b)
    state |= {"cu_q": cu_q, "cu_kv": cu_kv}
    # the same lengths on the device, for the plain form
    state["dev_q"] = torch.tensor(cu_q, device="cuda")
    state["dev_kv"] = torch.tensor(cu_kv, device="cuda")

    def packed(total, heads):
        if case["token_major"]:
            return _normal((total, heads, d), gen).transpose(0, 1)
        return _normal((heads, total, d), gen)

    state["q"], state["k"], state["v"] = packed(cu_q[-1], hq), packed(cu_kv[-1], hkv), packed(cu_kv[-1], hkv)
    if case["op"] == "train":
        state["dout"] = packed(cu_q[-1], hq)
        out, state["lse"] = _forward(state)
        state["out"] = torch.empty_like(state["q"]).copy_(out)
    return state


def _padding(cu, longest):
    """For packed rows cu[i] .. cu[i + 1]: the row of each padded place [n, longest], whether it is one, and the padded place of each row [total]."""
    n = cu.numel() - 1
    at = torch.arange(longest, device=cu.device)
    rows = cu[:-1, None] + at
    real = rows < cu[1:, None]
    return rows, real, n


def _places(cu, longest, total):
    row = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq * longest + row - cu[seq]


def _padded(x, cu, longest):
    """[heads, total, d] packed -> [n, heads, longest, d] in 32 bits, zeros behind each sequence."""
    rows, real, n = _padding(cu, longest)
    y = x[:, rows.clamp(max=x.shape[1] - 1)].float()
    return torch.where(real[None, :, :, None], y, 0.0).transpose(0, 1)


def _packed(y, cu, total):
    """The inverse of _padded."""
    n, heads, longest, d = y.shape
    return y.transpose(0, 1).reshape(heads, n * longest, d)[:, _places(cu, longest, total)]


def _scores(state):
    """(grouped q [n, Hkv, G * Lq, d], k, v [n, Hkv, Lkv, d], masked scaled scores [n, Hkv, G, Lq, Lkv])."""
    case = state["case"]
    pairs = _pairs_of(case["lens"])
    lq, lkv = max(a for a, _ in pairs), max(b for _, b in pairs)
    n, hkv, g, d = len(pairs), case["hkv"], case["hq"] // case["hkv"], case["d"]
    q = _padded(state["q"], state["dev_q"], lq).reshape(n, hkv, g * lq, d)
    k, v = _padded(state["k"], state["dev_kv"], lkv), _padded(state["v"], state["dev_kv"], lkv)
    s = (q @ k.transpose(-1, -2)).mul_(state["scale"]).view(n, hkv, g, lq, lkv)
    len_q, len_kv = state["dev_q"].diff()[:, None, None], state["dev_kv"].diff()[:, None, None]
    row, key = torch.arange(lq, device=s.device)[:, None], torch.arange(lkv, device=s.device)
    seen = (key < len_kv) & (row < len_q)
    if case["causal"]:
        seen = seen & (key <= row + len_kv - len_q)
    s.masked_fill_(~seen[:, None, None], -math.inf)
    return q, k, v, s


def _forward(state):
    q, k, v, s = _scores(state)
    n, hkv, g, lq, lkv = s.shape
    hq, total = hkv * g, state["q"].shape[1]
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)  # a row that sees nothing
    p = s.sub_(top).exp_()
    norm = p.sum(-1, keepdim=True)
    out = (p.view(n, hkv, g * lq, lkv) @ v).view(n, hkv, g, lq, -1) / torch.where(norm == 0, 1.0, norm)
    lse = (top + norm.log()).view(n, hq, lq, 1)
    return (_packed(out.reshape(n, hq, lq, -1), state["dev_q"], total).to(torch.bfloat16),
            _packed(lse, state["dev_q"], total).squeeze(-1))


def _backward(state):
    q, k, v, s = _scores(state)
    n, hkv, g, lq, lkv = s.shape
    d, hq = q.shape[-1], hkv * g
    total_q, total_kv = state["q"].shape[1], state["k"].shape[1]
    lse = _padded(state["lse"][..., None], state["dev_q"], lq).view(n, hkv, g, lq, 1)
    out = _padded(state["out"], state["dev_q"], lq).reshape(n, hkv, g * lq, d)
    dout = _padded(state["dout"], state["dev_q"], lq).reshape(n, hkv, g * lq, d)
    p = s.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_().view(n, hkv, g * lq, lkv)
    dv = p.transpose(-1, -2) @ dout
    ds = (dout @ v.transpose(-1, -2)).sub_((dout * out).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * state["scale"]
    dk = (ds.transpose(-1, -2) @ q) * state["scale"]
    return (_packed(dq.reshape(n, hq, lq, d), state["dev_q"], total_q).to(torch.bfloat16),
            _packed(dk, state["dev_kv"], total_kv).to(torch.bfloat16),
            _packed(dv, state["dev_kv"], total_kv).to(torch.bfloat16))


def _decode(state):
    case = state["case"]
    b, t, hkv, g, d = case["batch"], case["tokens"], case["hkv"], case["hq"] // case["hkv"], case["d"]
    q = state["q"].float().reshape(b, hkv, g * t, d)
    # the prefix: all requests' rows of a key head against keys that are there once
    first = q.transpose(0, 1).reshape(hkv, b * g * t, d) @ state["k_prefix"].float().transpose(-1, -2)
    first = first.view(hkv, b, g, t, case["prefix"]).transpose(0, 1)
    rest = (q @ state["k_suffix"].float().transpose(-1, -2)).view(b, hkv, g, t, case["suffix"])
    key = torch.arange(case["suffix"], device=q.device)
    ends = state["lens"][:, None] - t + 1 + torch.arange(t, device=q.device)  # [b, t]
    rest = rest.masked_fill((key >= ends[:, :, None])[:, None, None], -math.inf)
    s = torch.cat([first, rest], -1).mul_(state["scale"])
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    p = p / p.sum(-1, keepdim=True)
    mine = p[..., case["prefix"]:].reshape(b, hkv, g * t, case["suffix"]) @ state["v_suffix"].float()
    shared = p[..., :case["prefix"]].transpose(0, 1).reshape(hkv, b * g * t, case["prefix"]) @ state["v_prefix"].float()
    out = mine + shared.view(hkv, b, g * t, d).transpose(0, 1)
    return out.reshape(b, hkv * g, t, d).to(torch.bfloat16)


def run(state):
    op = state["case"]["op"]
    if own:
        import block_sparse_attention_15_b200 as vsa

        if op == "prompt":
            return vsa.dense_attn_varlen(state["q"], state["k"], state["v"], state["cu_q"], state["cu_kv"],
                                         causal=state["case"]["causal"], return_lse=True)
        if op == "train":
            return vsa.dense_attn_varlen_backward(state["q"], state["k"], state["v"], state["out"], state["dout"], state["lse"],
                                                  state["cu_q"], state["cu_kv"], causal=state["case"]["causal"])
        return vsa.shared_prefix_attn(state["q"], state["k_prefix"], state["v_prefix"], state["k_suffix"], state["v_suffix"],
                                      state["lens"])
    return _forward(state) if op == "prompt" else _backward(state) if op == "train" else _decode(state)


def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "decode":
        b, t, p = case["batch"], case["tokens"], case["prefix"]
        mean = (t + case["suffix"]) / 2  # lengths are spread evenly from `tokens` to `suffix`
        kv = 2 * hkv * d * 2 * (p + b * mean)
        return {"bytes": int(kv + 2 * b * hq * t * d * 2 + 4 * b), "flops": int(4 * d * b * hq * t * (p + mean))}
    pairs = _pairs_of(case["lens"])
    tq, tkv = sum(a for a, _ in pairs), sum(b for _, b in pairs)
    seen = sum(_visible(a, b, case["causal"]) for a, b in pairs) * hq
    if case["op"] == "prompt":
        return {"bytes": 2 * d * (2 * hq * tq + 2 * hkv * tkv) + 4 * hq * tq, "flops": 4 * d * seen}
    return {"bytes": 2 * d * (4 * hq * tq + 4 * hkv * tkv) + 4 * hq * tq, "flops": 10 * d * seen}


def _attend64(q, k, v, scale, seen):
    """One head in 64 bits: probabilities, output and log-sum-exp; `seen` [rows, keys] or None."""
    s = q @ k.T * scale
    if seen is not None:
        s = torch.where(seen, s, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(torch.isinf(s), 0.0, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[:, None]))
    return p, p @ v, lse


def exact(case, seed):
    state = prepare(case, seed)
    wide = {n: x.double() for n, x in state.items() if isinstance(x, torch.Tensor) and x.dtype == torch.bfloat16}
    group, scale = case["hq"] // case["hkv"], 1.0 / math.sqrt(case["d"])
    if case["op"] == "decode":
        out = torch.zeros(wide["q"].shape, dtype=torch.float64, device="cuda")
        t = case["tokens"]
        for b, n in enumerate(state["lens"].tolist()):
            keys = torch.arange(case["prefix"] + n, device="cuda")
            seen = keys < case["prefix"] + n - t + 1 + torch.arange(t, device="cuda")[:, None]
            for h in range(case["hq"]):
                k = torch.cat([wide["k_prefix"][h // group], wide["k_suffix"][b, h // group, :n]])
                v = torch.cat([wide["v_prefix"][h // group], wide["v_suffix"][b, h // group, :n]])
                out[b, h] = _attend64(wide["q"][b, h], k, v, scale, seen)[1]
        return out
    rows, cols = state["cu_q"], state["cu_kv"]
    out, lse = torch.zeros_like(wide["q"]), torch.zeros(wide["q"].shape[:2], dtype=torch.float64, device="cuda")
    grads = {n: torch.zeros_like(wide[n]) for n in "qkv"}
    for i in range(len(rows) - 1):
        a, b = slice(rows[i], rows[i + 1]), slice(cols[i], cols[i + 1])
        lq, lkv = rows[i + 1] - rows[i], cols[i + 1] - cols[i]
        seen = torch.ones(lq, lkv, dtype=torch.bool, device="cuda").tril(lkv - lq) if case["causal"] else None
        for h in range(case["hq"]):
            q, k, v = wide["q"][h, a], wide["k"][h // group, b], wide["v"][h // group, b]
            p, o, l = _attend64(q, k, v, scale, seen)
            out[h, a], lse[h, a] = o, l
            if case["op"] == "train":
                do = wide["dout"][h, a]
                ds = p * (do @ v.T - (do * o).sum(-1, keepdim=True))
                grads["q"][h, a] = ds @ k * scale
                grads["k"][h // group, b] += ds.T @ q * scale
                grads["v"][h // group, b] += p.T @ do
    return (grads["q"], grads["k"], grads["v"]) if case["op"] == "train" else (out, lse)
