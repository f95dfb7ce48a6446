"""Cases of the attention operators: a whole prompt (``gdn_attn_fwd``), a chunk of new tokens or one token over a
paged cache (``gdn_attn_paged_fwd``), and the write of new keys and values into the pages (``gdn_kv_cache_append``).

``run`` computes a case through this package's entry points when ``own`` is true, and from elementary torch
operations in 32 bits otherwise.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one short question: a single small call, where latency is all that counts
        _prompt("prompt_33", seqs=1, tokens=33, heads=16, kv_heads=2),
        # an ordinary prefill batch of four equal prompts
        _prompt("prompt_4x2048", seqs=4, tokens=2048, heads=32, kv_heads=8),
        # the longest single prompt of the benchmark's own length
        _prompt("prompt_32768", seqs=1, tokens=32768, heads=16, kv_heads=2),
        # eight requests of very different odd lengths (one of one token, one empty) packed without padding, 48 heads
        _prompt("prompt_packed", seqs=8, tokens=12001, heads=48, kv_heads=8, packed=True),
        # 32-bit inputs, one key/value head per query head, q, k and v as slices of one projection's output
        _prompt("prompt_f32_qkv", seqs=2, tokens=1023, heads=16, kv_heads=16, dim=64, dtype="f32", sliced=True),
        # one user, one token, a short conversation: the smallest decode step
        _paged("decode_1x300", seqs=1, kv=300, heads=16, kv_heads=2, page=16),
        # a full serving batch, one token each, cached lengths from a few hundred to 4096
        _paged("decode_256", seqs=256, kv=4096, heads=32, kv_heads=8, page=16, ragged=True),
        # one user with a very long document: one token against 131072
        _paged("decode_131072", seqs=1, kv=131072, heads=16, kv_heads=2, page=64),
        # a prompt's next 512 tokens over what is already cached
        _paged("chunk_512", seqs=1, kv=32768, heads=32, kv_heads=8, page=64, new=512, chunks=1),
        # a serving step that mixes two prompt chunks with fourteen one-token sequences, heads of 64
        _paged("step_mixed", seqs=16, kv=8192, heads=32, kv_heads=4, dim=64, page=32, new=500, chunks=2, ragged=True),
        # the cache write of that full serving batch: one token for each of 256 sequences
        _append("append_256", seqs=256, new=1, kv=1024, kv_heads=8, page=16),
        # the cache write of a long prompt
        _append("append_32768", seqs=1, new=32768, kv=32768, kv_heads=8, page=64),
    ]


def _prompt(name, seqs, tokens, heads, kv_heads, dim=128, dtype="bf16", packed=False, sliced=False, mix=0):
    """tokens: of each sequence, or of all of them together where they are packed."""
    c = {"op": "prompt", "dtype": dtype, "seqs": seqs, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
         "packed": packed, "sliced": sliced, "mix": mix}
    return c if name is None else {**c, "name": name}


def _paged(name, seqs, kv, heads, kv_heads, page, dim=128, dtype="bf16", new=1, chunks=0, ragged=False, mix=0):
    """kv: the longest cached length, the new tokens among it; the first `chunks` sequences bring up to `new` tokens, the others one."""
    c = {"op": "paged", "dtype": dtype, "seqs": seqs, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "new": new, "chunks": chunks, "ragged": ragged, "mix": mix}
    return c if name is None else {**c, "name": name}


def _append(name, seqs, new, kv, kv_heads, page, dim=128, dtype="bf16", ragged=False, mix=0):
    c = {"op": "append", "dtype": dtype, "seqs": seqs, "new": new, "kv": kv, "kv_heads": kv_heads, "dim": dim, "page": page,
         "ragged": ragged, "mix": mix}
    return c if name is None else {**c, "name": name}


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
        heads = kv_heads * rng.choice((1, 2, 4, 5, 6, 8, 16))
        dim, dtype = rng.choice((64, 128, 128)), rng.choice(("bf16",) * 4 + ("f32",))
        page, mix = rng.choice((16, 32, 48, 64, 128)), rng.randrange(1 << 20)
        op = rng.choice(("prompt", "prompt", "paged", "paged", "append"))
        if op == "prompt":
            packed = rng.random() < 0.5
            seqs = _log_between(rng, 1, 12)
            c = _prompt(None, seqs, _log_between(rng, 1, 16384), heads, kv_heads, dim, dtype, packed, rng.random() < 0.3, mix)
        elif op == "paged":
            seqs, kv = _log_between(rng, 1, 256), _log_between(rng, 1, 131072)
            new = _log_between(rng, 1, 1024)
            chunks = rng.choice((0, 0, min(seqs, rng.randint(1, 3))))
            c = _paged(None, seqs, kv, heads, kv_heads, page, dim, dtype, min(new, kv), chunks, rng.random() < 0.7, mix)
        else:
            kv = _log_between(rng, 1, 16384)
            c = _append(None, _log_between(rng, 1, 256), _log_between(rng, 1, kv), kv, kv_heads, page, dim, dtype, rng.random() < 0.7, mix)
        if 3072 in (heads * dim, kv_heads * dim, (heads + 2 * kv_heads) * dim, *c.values()):
            continue  # not a width that this library is used at
        w = work(c)
        # 32-bit products run at a fraction of the 16-bit rate, and the scores of a padded batch have to fit the card
        flops = w["flops"] * (16 if dtype == "f32" else 1)
        if flops <= 4e12 and w["bytes"] <= 2e9 and _scores(c) <= 8e9 and _pool(c) <= 4e9:
            return c


def _scores(c):
    """Elements of the score matrix and of the gathered keys when every sequence is padded to the longest."""
    if c["op"] == "append":
        return 0
    q, kv = _lengths(c)
    return len(q) * max(kv, default=0) * max(max(q, default=0) * c["heads"], 2 * c["kv_heads"] * c["dim"])


def _pool(c):
    """Bytes of one cache."""
    return 0 if c["op"] == "prompt" else _pages(c) * c["page"] * c["kv_heads"] * c["dim"] * (4 if c["dtype"] == "f32" else 2)


def _lengths(c):
    """(new tokens, keys) of each sequence, from the case alone."""
    rng = random.Random(c["mix"])
    n = c["seqs"]
    if c["op"] == "prompt":
        if not c["packed"]:
            return [c["tokens"]] * n, [c["tokens"]] * n
        weights = [rng.random() ** 2 + 1e-3 for _ in range(n)]
        q = [int(c["tokens"] * w / sum(weights)) for w in weights]
        if n >= 6 and c["tokens"] >= 16 * n:
            q[1], q[4] = 0, 1
        q[-1] += c["tokens"] - sum(q)
        return q, q
    if c["op"] == "append":
        q = [max(1, int(c["new"] * rng.uniform(0.2, 1))) if c["ragged"] else c["new"] for _ in range(n)]
        return q, [max(a, int(c["kv"] * rng.uniform(0.2, 1))) if c["ragged"] else max(a, c["kv"]) for a in q]
    kv = [max(1, int(c["kv"] * rng.uniform(0.05, 1))) if c["ragged"] else c["kv"] for _ in range(n)]
    kv[0] = c["kv"]
    q = [min(kv[i], max(1, int(c["new"] * rng.uniform(0.5, 1)) if c["ragged"] else c["new"])) if i < c["chunks"] else 1 for i in range(n)]
    return q, kv


def _width(c):
    """Pages in a row of the block table."""
    return -(-max(_lengths(c)[1]) // c["page"])


def _pages(c):
    """Pages of the pool: what the sequences hold, and a few free ones."""
    return sum(-(-n // c["page"]) for n in _lengths(c)[1]) + 7


def work(case):
    c, size = case, 4 if case["dtype"] == "f32" else 2
    q, kv = _lengths(c)
    row = c["kv_heads"] * c["dim"] * size
    if c["op"] == "append":
        return {"bytes": 4 * sum(q) * row + 4 * (2 * len(q) + sum(-(-n // c["page"]) for n in q)), "flops": 0}
    pairs = sum(a * (2 * b - a + 1) // 2 for a, b in zip(q, kv))
    out = sum(q) * c["heads"] * (2 * c["dim"] * size + 4)  # q read, o and the log-sum-exp written
    table = 0 if c["op"] == "prompt" else 4 * sum(-(-n // c["page"]) + 1 for n in kv)
    return {"bytes": 2 * sum(kv) * row + out + table, "flops": 4 * c["dim"] * c["heads"] * pairs}


# ---- inputs ---------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    c, dev, dt = case, torch.device("cuda"), _DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=dt, device=dev).normal_(0.0, std, generator=gen)

    q_lens, kv_lens = _lengths(c)
    n, total, hkv, d = c["seqs"], sum(q_lens), c["kv_heads"], c["dim"]
    cu = [sum(q_lens[:i]) for i in range(n + 1)]
    uniform = len(set(q_lens)) == 1 and not c.get("packed")
    s = {"case": c, "scale": d ** -0.5, "uniform": uniform,
         "cu": None if uniform else torch.tensor(cu, dtype=torch.int32, device=dev),
         "kv_lens": torch.tensor(kv_lens, dtype=torch.int32, device=dev)}
    lead = (n, q_lens[0]) if uniform else (1, total)
    # where each new token's row is in the padded batch [n, longest]: what the plain form gathers and scatters by
    longest = max(max(q_lens), 1)
    s["slot"] = torch.cat([torch.arange(m, device=dev) + i * longest for i, m in enumerate(q_lens)])
    s["longest"] = longest
    s["pos"] = torch.arange(longest, device=dev)[None] + torch.tensor([b - a for a, b in zip(q_lens, kv_lens)], device=dev)[:, None]
    if c["op"] != "append":
        # queries a little above unit size, so that some rows look at few keys and some at many
        if c.get("sliced"):
            qkv = normal(*lead, (c["heads"] + 2 * hkv) * d, std=1.5)
            s["qkv"] = qkv
        else:
            s["q"] = normal(*lead, c["heads"], d, std=2.0)
    if c["op"] != "paged" and not c.get("sliced"):
        s["k"], s["v"] = normal(*lead, hkv, d), normal(*lead, hkv, d)
    if c["op"] != "prompt":
        # a pool in use: the pages lie in any order, and those that nobody holds keep an earlier request's values
        pool = _pages(c)
        s["k_cache"], s["v_cache"] = normal(pool, c["page"], hkv, d), normal(pool, c["page"], hkv, d)
        perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
        held = torch.tensor([-(-m // c["page"]) for m in kv_lens], device=dev)
        col = torch.arange(_width(c), device=dev)[None]
        first = (held.cumsum(0) - held)[:, None]
        s["table"] = torch.where(col < held[:, None], perm[(first + col).clamp_(max=pool - 1)], 0).to(torch.int32).contiguous()
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------
def _split(s):
    c = s["case"]
    if "qkv" not in s:
        return s["q"], s["k"], s["v"]
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    x = s["qkv"].unflatten(-1, (h + 2 * g, d))
    return x[:, :, :h], x[:, :, h:h + g], x[:, :, h + g:]


def run(state):
    c = state["case"]
    if own:
        from chunkwise_gated_delta_gdn_gb300 import gdn

        if c["op"] == "prompt":
            q, k, v = _split(state)
            return gdn.gdn_attn_fwd(q, k, v, scale=state["scale"], cu_seqlens=state["cu"])
        if c["op"] == "paged":
            return gdn.gdn_attn_paged_fwd(state["q"], state["k_cache"], state["v_cache"], state["table"], state["kv_lens"],
                                          scale=state["scale"], cu_seqlens=state["cu"])
        gdn.gdn_kv_cache_append(state["k"], state["v"], state["k_cache"], state["v_cache"], state["table"], state["kv_lens"],
                                cu_seqlens=state["cu"])
        return state["k_cache"], state["v_cache"]
    if c["op"] == "append":
        return _plain_append(state)
    if c["op"] == "prompt":
        q, k, v = _split(state)
        k, v = _padded(state, k), _padded(state, v)
    else:
        q, k, v = state["q"], _gathered(state, state["k_cache"]), _gathered(state, state["v_cache"])
    return _plain_attention(state, q, k, v)


def _padded(s, x):
    """Packed or batched rows [.., heads, dim] as 32-bit [sequences, longest, heads, dim]."""
    x = x.float()
    if s["uniform"]:
        return x
    out = torch.zeros(s["case"]["seqs"] * s["longest"], *x.shape[2:], device=x.device)
    out[s["slot"]] = x[0]
    return out.unflatten(0, (s["case"]["seqs"], s["longest"]))


def _gathered(s, cache):
    return cache[s["table"].long()].flatten(1, 2).float()


def _plain_attention(s, q, k, v):
    dt, hkv = q.dtype, k.shape[2]
    lead = q.shape[:2]
    q = _padded(s, q)
    n, t, h, d = q.shape
    q = q.unflatten(2, (hkv, h // hkv)).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).unflatten(2, (-1, t))
    key = torch.arange(k.shape[1], device=q.device)
    seen = (key <= s["pos"][:, :, None]) & (key < s["kv_lens"][:, None, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    v = torch.where((key < s["kv_lens"][:, None])[:, :, None, None], v, 0.0)
    o = torch.matmul(weights.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (-1, t))
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n * t, h, d)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(n * t, h)
    if not s["uniform"]:
        o, lse = o[s["slot"]], lse[s["slot"]]
    return o.to(dt).reshape(*lead, h, d), lse.reshape(*lead, h)


def _plain_append(s):
    page = s["case"]["page"]
    seq = torch.div(s["slot"], s["longest"], rounding_mode="floor")
    pos = s["pos"].reshape(-1)[s["slot"]]
    where = s["table"][seq, torch.div(pos, page, rounding_mode="floor")].long(), pos % page
    s["k_cache"][where] = s["k"].flatten(0, 1)
    s["v_cache"][where] = s["v"].flatten(0, 1)
    return s["k_cache"], s["v_cache"]


# ---- the definition in 64 bits --------------------------------------------------------------------------------------
def exact(case, seed):
    s, c = prepare(case, seed), case
    if work(c)["flops"] > 5e12:
        return None
    q_lens, kv_lens = _lengths(c)
    page, hkv, d = c["page"] if "page" in c else 0, c["kv_heads"], c["dim"]
    if c["op"] == "append":
        out = [s["k_cache"].double(), s["v_cache"].double()]
        for cache, new in zip(out, (s["k"], s["v"])):
            new, at = new.double().reshape(-1, hkv, d), 0
            for i, (a, b) in enumerate(zip(q_lens, kv_lens)):  # a sequence's pages in order, its last rows replaced, put back
                rows = s["table"][i, :-(-b // page)].long()
                held = cache[rows]
                held.view(-1, hkv, d)[b - a:b] = new[at:at + a]
                cache[rows] = held
                at += a
        return tuple(out)
    q, k, v = _split(s) if c["op"] == "prompt" else (s["q"], None, None)
    lead, h, group = q.shape[:2], c["heads"], c["heads"] // hkv
    q = q.reshape(-1, h, d)
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    at = 0
    for i, (a, b) in enumerate(zip(q_lens, kv_lens)):
        if c["op"] == "prompt":
            ki, vi = k.reshape(-1, hkv, d)[at:at + a].double(), v.reshape(-1, hkv, d)[at:at + a].double()
        else:
            rows = s["table"][i, :-(-b // page)].long()
            ki, vi = s["k_cache"][rows].reshape(-1, hkv, d)[:b].double(), s["v_cache"][rows].reshape(-1, hkv, d)[:b].double()
        for head in range(hkv):
            for lo in range(0, a, 1024):  # query rows a block at a time, against the keys that its last row sees
                hi = min(a, lo + 1024)
                end = b - a + hi
                x = q[at + lo:at + hi, head * group:(head + 1) * group].double()
                sc = torch.einsum("tgd,kd->tgk", x, ki[:end, head]) * s["scale"]
                later = torch.arange(end, device=q.device)[None] > torch.arange(b - a + lo, end, device=q.device)[:, None]
                lg = torch.logsumexp(sc.masked_fill_(later[:, None], -math.inf), -1)
                o[at + lo:at + hi, head * group:(head + 1) * group] = torch.einsum("tgk,kd->tgd", (sc - lg[..., None]).exp_(), vi[:end, head])
                lse[at + lo:at + hi, head * group:(head + 1) * group] = lg
        at += a
    return o.reshape(*lead, h, d), lse.reshape(*lead, h)
