"""Cases of the operators around a key/value cache held in 8 bits: rotary positions of queries and keys (``gdn_rope_fwd``,
``gdn_rope_bwd``), the quantising write of new keys and values into the pages (``gdn_kv_cache_append_fp8``), attention over
such pages (``gdn_attn_paged_fp8_fwd``), and the copy of pages when a sequence forks or a pool is put in order
(``gdn_kv_cache_copy_pages``).

A cache's values are 8-bit floating point (4 exponent, 3 mantissa bits) times a 32-bit scale for each block of 16 tokens and
head.  ``run`` computes a case through this package's entry points when ``own`` is true, and from elementary torch operations
in 32 bits otherwise.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BLOCK = 16   # tokens of a cache that share a scale
_TOP = 448.0  # the largest 8-bit value


# ---- the cases ------------------------------------------------------------------------------------------------------
def listed():
    return [
        # the queries and keys of a serving batch's one new token each, far along in their sequences: latency
        _rope("rope_decode_256", seqs=256, tokens=1, heads=32, kv_heads=8, past=4095, ragged=True),
        # a long prompt, q and k as slices of one projection's output
        _rope("rope_prompt_32768", seqs=1, tokens=32768, heads=32, kv_heads=8, sliced=True),
        # gradients of packed prompts in 32 bits: part of each head rotated, neighbours paired, scaled for long contexts
        _rope("rope_packed_grad", seqs=8, tokens=12001, heads=16, kv_heads=16, dim=64, dtype="f32", packed=True, rot=32,
              interleaved=True, stretch=8.0, backward=True),
        # the cache write of a serving step: one token for each of 256 sequences, most of them into a block that is held in part
        _append("append8_256", seqs=256, new=1, kv=4096, kv_heads=8, page=16, ragged=True),
        # the cache write of a long prompt
        _append("append8_32768", seqs=1, new=32768, kv=32768, kv_heads=8, page=64),
        # one user, one token, a short conversation: the smallest decode step
        _paged("decode8_1x300", seqs=1, kv=300, heads=16, kv_heads=2, page=16),
        # a full serving batch, one token each, cached lengths from a few hundred to 4096
        _paged("decode8_256", seqs=256, kv=4096, heads=32, kv_heads=8, page=16, ragged=True),
        # one user with a very long document: one token against 131072
        _paged("decode8_131072", seqs=1, kv=131072, heads=16, kv_heads=2, page=64),
        # a prompt's next 512 tokens over what is already cached
        _paged("chunk8_512", seqs=1, kv=32768, heads=32, kv_heads=8, page=64, new=512, chunks=1),
        # a serving step that mixes two prompt chunks with fourteen one-token sequences, heads of 64
        _paged("step8_mixed", seqs=16, kv=8192, heads=32, kv_heads=4, dim=64, page=32, new=500, chunks=2, ragged=True),
        # 32 sequences fork: the last page of each is copied before the two go their own ways
        _copy("copy_fork_32", pages=32, kv_heads=8, page=64),
        # a pool put in order: thousands of pages of an 8-bit cache, with their scales
        _copy("copy_pool_4096", pages=4096, kv_heads=8, page=64, dtype="e4m3"),
    ]


def _named(name, c):
    return c if name is None else {**c, "name": name}


def _rope(name, seqs, tokens, heads, kv_heads, dim=128, dtype="bf16", packed=False, sliced=False, ragged=False, past=0, rot=0,
          interleaved=False, stretch=1.0, backward=False, mix=0):
    """tokens: of each sequence, or of all of them together where they are packed; past: the most that is cached before them;
    rot: leading elements of a head that turn (0: all); stretch: of the positions' range."""
    return _named(name, {"op": "rope", "dtype": dtype, "seqs": seqs, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                         "packed": packed, "sliced": sliced, "ragged": ragged, "past": past, "rot": rot or dim,
                         "interleaved": interleaved, "stretch": stretch, "backward": backward, "mix": mix})


def _append(name, seqs, new, kv, kv_heads, page, dim=128, dtype="bf16", ragged=False, mix=0):
    return _named(name, {"op": "append", "dtype": dtype, "seqs": seqs, "new": new, "kv": kv, "kv_heads": kv_heads, "dim": dim,
                         "page": page, "ragged": ragged, "mix": mix})


def _paged(name, seqs, kv, heads, kv_heads, page, dim=128, new=1, chunks=0, ragged=False, mix=0):
    """kv: the longest cached length, the new tokens among it; the first `chunks` sequences bring up to `new` tokens, the others one."""
    return _named(name, {"op": "paged", "dtype": "bf16", "seqs": seqs, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                         "page": page, "new": new, "chunks": chunks, "ragged": ragged, "mix": mix})


def _copy(name, pages, kv_heads, page, dim=128, dtype="bf16"):
    return _named(name, {"op": "copy", "dtype": dtype, "pages": pages, "kv_heads": kv_heads, "page": page, "dim": dim})


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
        heads = kv_heads * rng.choice((1, 2, 4, 5, 6, 8, 16))
        dim, dtype = rng.choice((64, 128, 128)), rng.choice(("bf16",) * 4 + ("f32",))
        page, mix = rng.choice((16, 32, 48, 64, 128)), rng.randrange(1 << 20)
        op = rng.choice(("rope", "append", "paged", "paged", "copy"))
        if op == "rope":
            seqs, packed = _log_between(rng, 1, 256), rng.random() < 0.5
            c = _rope(None, seqs, _log_between(rng, 1, 32768 if packed else max(1, 32768 // seqs)), heads, kv_heads, dim, dtype, packed,
                      rng.random() < 0.3, rng.random() < 0.5, _log_between(rng, 1, 131072) - 1, 16 * rng.randint(1, dim // 16),
                      rng.random() < 0.5, rng.choice((1.0, 1.0, 4.0, 8.0)), rng.random() < 0.3, mix)
        elif op == "append":
            kv = _log_between(rng, 1, 16384)
            c = _append(None, _log_between(rng, 1, 256), _log_between(rng, 1, kv), kv, kv_heads, page, dim, dtype, rng.random() < 0.7, mix)
        elif op == "paged":
            seqs, kv = _log_between(rng, 1, 256), _log_between(rng, 1, 131072)
            new = _log_between(rng, 1, 1024)
            chunks = rng.choice((0, 0, min(seqs, rng.randint(1, 3))))
            c = _paged(None, seqs, kv, heads, kv_heads, page, dim, min(new, kv), chunks, rng.random() < 0.7, mix)
        else:
            c = _copy(None, _log_between(rng, 1, 4096), kv_heads, page, dim, rng.choice(("bf16", "e4m3", "e4m3", "f32")))
        w = work(c)
        # no more work than the largest listed case's; a padded batch's scores and gathered keys have to fit the card, a pool three times
        if w["flops"] <= 2.7e11 and w["bytes"] <= 1.07e9 and _padded_size(c) <= 8e9 and _pool(c) <= 4e9:
            return c


def _padded_size(c):
    """Elements of the largest intermediate tensor when every sequence is padded to the longest."""
    if c["op"] == "copy":
        return 0
    q, kv = _lengths(c)
    if c["op"] == "paged":
        return len(q) * max(kv, default=0) * max(max(q, default=0) * c["heads"], 2 * c["kv_heads"] * c["dim"])
    heads = c["kv_heads"] if c["op"] == "append" else c["heads"] + c["kv_heads"]
    return 4 * len(q) * (max(q, default=0) + 2 * _BLOCK) * heads * c["dim"]


def _pool(c):
    """Elements of the two caches."""
    return 0 if c["op"] == "rope" else 2 * _pages(c) * c["page"] * c["kv_heads"] * c["dim"]


def _lengths(c):
    """(new tokens, keys) of each sequence, from the case alone."""
    rng = random.Random(c["mix"])
    n = c["seqs"]
    if c["op"] == "rope":
        if c["packed"]:
            weights = [rng.random() ** 2 + 1e-3 for _ in range(n)]
            q = [int(c["tokens"] * w / sum(weights)) for w in weights]
            if n >= 6 and c["tokens"] >= 16 * n:
                q[1], q[4] = 0, 1
            q[-1] += c["tokens"] - sum(q)
        else:
            q = [c["tokens"]] * n
        return q, [a + (int(c["past"] * rng.random()) if c["ragged"] else c["past"]) for a in q]
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
    """Pages of the pool: what the sequences hold, and a few free ones; of a copy, its sources, its destinations and others."""
    return 2 * c["pages"] + 7 if c["op"] == "copy" else sum(-(-n // c["page"]) for n in _lengths(c)[1]) + 7


def _size(c):
    return {"bf16": 2, "f32": 4, "e4m3": 1}[c["dtype"]]


def work(case):
    c = case
    if c["op"] == "copy":
        page = c["page"] * c["kv_heads"] * (c["dim"] * _size(c) + (4 / _BLOCK if c["dtype"] == "e4m3" else 0))
        return {"bytes": 4 * c["pages"] * page + 8 * c["pages"], "flops": 0}
    q, kv = _lengths(c)
    if c["op"] == "rope":
        rows = sum(q) * (c["heads"] + c["kv_heads"])
        return {"bytes": 2 * rows * c["dim"] * _size(c) + 4 * len(q) + 2 * c["rot"], "flops": 3 * rows * c["rot"]}
    row = c["kv_heads"] * c["dim"]
    held = sum(-(-n // c["page"]) for n in kv)
    if c["op"] == "append":  # each new token read and written in 8 bits, and a scale for each block that it reaches
        blocks = sum((b - 1) // _BLOCK - (b - a) // _BLOCK + 1 for a, b in zip(q, kv))
        return {"bytes": 2 * sum(q) * row * (_size(c) + 1) + 8 * blocks * c["kv_heads"] + 4 * (2 * len(q) + held), "flops": 0}
    pairs = sum(a * (2 * b - a + 1) // 2 for a, b in zip(q, kv))
    scales = 8 * c["kv_heads"] * sum(-(-n // _BLOCK) for n in kv)
    out = sum(q) * c["heads"] * (4 * c["dim"] + 4)  # q read, o and the log-sum-exp written
    return {"bytes": 2 * sum(kv) * row + scales + out + 4 * (held + len(q)), "flops": 4 * c["dim"] * c["heads"] * pairs}


# ---- inputs ---------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dt=_DTYPES[case["dtype"]]):
        return torch.empty(shape, dtype=dt, device=dev).normal_(0.0, std, generator=gen)

    hkv, d, s = c["kv_heads"], c["dim"], {"case": case}
    if c["op"] != "rope":
        # a pool in use: the pages lie in any order, and those that nobody holds keep an earlier request's values
        pool, page = _pages(c), c["page"]
        perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
        for name in ("k", "v"):
            if c["op"] == "copy" and c["dtype"] != "e4m3":
                s[name + "_cache"], s[name + "_scale"] = normal(pool, page, hkv, d), None
                continue
            codes = torch.empty((pool, page, hkv, d), dtype=torch.float8_e4m3fn, device=dev)
            scales = torch.empty((pool, page // _BLOCK, hkv), device=dev)
            for lo in range(0, pool, 1024):  # some tokens' rows are larger than others', as a network's are
                x = normal(min(1024, pool - lo), page, hkv, d, dt=torch.float32)
                x *= normal(x.shape[0], page, 1, 1, std=0.5, dt=torch.float32).exp_()
                x = x.unflatten(1, (-1, _BLOCK))
                scale = _fitting(x.abs().amax((2, 4)))
                codes[lo:lo + 1024] = (x / scale[:, :, None, :, None]).flatten(1, 2).to(torch.float8_e4m3fn)
                scales[lo:lo + 1024] = scale
            s[name + "_cache"], s[name + "_scale"] = codes, scales
        if c["op"] == "copy":
            s["src"], s["dst"] = perm[:c["pages"]].contiguous(), perm[c["pages"]:2 * c["pages"]].contiguous()
            return s
    q_lens, kv_lens = _lengths(c)
    n, total = c["seqs"], sum(q_lens)
    uniform = len(set(q_lens)) == 1 and not c.get("packed")
    lead = (n, q_lens[0]) if uniform else (1, total)
    cu = [sum(q_lens[:i]) for i in range(n + 1)]
    s["uniform"], s["longest"] = uniform, max(max(q_lens), 1)
    s["cu"] = None if uniform else torch.tensor(cu, dtype=torch.int32, device=dev)
    s["q_lens"], s["kv_lens"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (q_lens, kv_lens))
    # what the plain forms gather and scatter by: each new token's row in the padded batch [n, longest], and the rows' positions
    s["slot"] = torch.cat([torch.arange(m, device=dev) + i * s["longest"] for i, m in enumerate(q_lens)])
    s["pos"] = torch.arange(s["longest"], device=dev)[None] + (s["kv_lens"] - s["q_lens"])[:, None]
    s["first"] = torch.tensor(cu[:-1], device=dev)
    if c["op"] == "rope":
        s["inv_freq"], s["mscale"] = _frequencies(c["rot"], c["stretch"]).to(dev), 0.1 * math.log(c["stretch"]) + 1.0
        if c["sliced"]:
            s["qkv"] = normal(*lead, (c["heads"] + 2 * hkv) * d)
        else:
            s["q"], s["k"] = normal(*lead, c["heads"], d), normal(*lead, hkv, d)
        return s
    held = torch.tensor([-(-m // c["page"]) for m in kv_lens], device=dev)
    col = torch.arange(_width(c), device=dev)[None]
    first = (held.cumsum(0) - held)[:, None]
    s["table"] = torch.where(col < held[:, None], perm[(first + col).clamp_(max=pool - 1)], 0).to(torch.int32).contiguous()
    if c["op"] == "paged":
        # queries a little above unit size, so that some rows look at few keys and some at many
        s["q"], s["scale"] = normal(*lead, c["heads"], d, std=2.0), d ** -0.5
    else:
        s["k"], s["v"] = normal(*lead, hkv, d), normal(*lead, hkv, d)
    return s


def _frequencies(rot, stretch):
    """Angles per position of the pairs; with `stretch`, pairs that turn less than once in 4096 positions turn so much slower,
    those that turn more than 32 times as before, those between in part."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    turns = 4096 * freq / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (freq * keep + freq / stretch * (1 - keep)).float()


def _fitting(top):
    """The smallest power of two that brings values of magnitude `top` into the 8 bits' range; 2^-117 to 2^120."""
    part, power = torch.frexp(top)
    power = power - 9 + (2 * part > 1.75)
    power = torch.where(top == 0, -117, power).clamp(-117, 120)
    return ((power.to(torch.int32) + 127) << 23).view(torch.float32)


# ---- one pass -------------------------------------------------------------------------------------------------------
def _q_and_k(s):
    if "qkv" not in s:
        return s["q"], s["k"]
    h, g, d = s["case"]["heads"], s["case"]["kv_heads"], s["case"]["dim"]
    x = s["qkv"].unflatten(-1, (h + 2 * g, d))
    return x[:, :, :h], x[:, :, h:h + g]


def run(state):
    s, c = state, state["case"]
    if own:
        from chunkwise_gated_delta_gdn_gb300 import gdn

        if c["op"] == "rope":
            q, k = _q_and_k(s)
            turn = gdn.gdn_rope_bwd if c["backward"] else gdn.gdn_rope_fwd
            return turn(q, k, s["inv_freq"], interleaved=c["interleaved"], mscale=s["mscale"], kv_lens=s["kv_lens"], cu_seqlens=s["cu"])
        if c["op"] == "paged":
            return gdn.gdn_attn_paged_fp8_fwd(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["kv_lens"],
                                              scale=s["scale"], cu_seqlens=s["cu"])
        if c["op"] == "append":
            gdn.gdn_kv_cache_append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["kv_lens"],
                                        cu_seqlens=s["cu"])
        else:
            gdn.gdn_kv_cache_copy_pages(s["k_cache"], s["v_cache"], s["src"], s["dst"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if c["op"] == "rope":
        return _plain_rope(s)
    if c["op"] == "paged":
        return _plain_attention(s)
    if c["op"] == "append":
        _plain_append(s, s["k"], s["k_cache"], s["k_scale"])
        _plain_append(s, s["v"], s["v_cache"], s["v_scale"])
    else:
        src, dst = s["src"].long(), s["dst"].long()
        for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
            if s[name] is not None:
                x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
                x[dst] = x[src]
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    # far positions: an angle in 32 bits would be off by a hundredth
    angle = s["pos"].reshape(-1)[s["slot"]].double()[:, None] * s["inv_freq"].double()
    cos, sin = (s["mscale"] * angle.cos()).float()[:, None], (s["mscale"] * angle.sin()).float()[:, None]
    if c["backward"]:
        sin = -sin
    out = []
    for x in _q_and_k(s):
        y = x.float().flatten(0, 1)
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        turned = a * cos - b * sin, a * sin + b * cos
        turned = torch.stack(turned, -1).flatten(-2) if c["interleaved"] else torch.cat(turned, -1)
        out.append(torch.cat((turned, y[..., rot:]), -1).to(x.dtype).reshape(x.shape))
    return tuple(out)


def _plain_append(s, x, cache, scales):
    """Each block that new tokens reach, padded to the same number for each sequence: its scale grows to what the new rows need
    (a block that begins with them has no earlier one), the rows that it held are rounded to the new scale, the new ones too."""
    c = s["case"]
    page, hkv, d = c["page"], c["kv_heads"], c["dim"]
    past, end = (s["kv_lens"] - s["q_lens"]).long(), s["kv_lens"].long()
    blocks = (s["longest"] + 2 * _BLOCK - 2) // _BLOCK
    index = torch.div(past, _BLOCK, rounding_mode="floor")[:, None] + torch.arange(blocks, device=x.device)
    reached = index * _BLOCK < end[:, None]
    where = index.clamp(max=s["table"].shape[1] * (page // _BLOCK) - 1)
    flat = s["table"].gather(1, torch.div(where * _BLOCK, page, rounding_mode="floor")).long() * (page // _BLOCK) + where % (page // _BLOCK)
    pos = index[..., None] * _BLOCK + torch.arange(_BLOCK, device=x.device)
    new = (pos >= past[:, None, None]) & (pos < end[:, None, None])
    row = (s["first"][:, None, None] + pos - past[:, None, None]).clamp(0, max(x.shape[0] * x.shape[1] - 1, 0))
    values = torch.where(new[..., None, None], x.flatten(0, 1)[row].float(), 0.0)
    need = _fitting(values.abs().amax((2, 4)))
    flat_scales, codes = scales.view(-1, hkv), cache.view(torch.uint8).view(-1, _BLOCK, hkv * d)
    holds = (index * _BLOCK < past[:, None])[..., None]
    old = torch.where(holds, flat_scales[flat], 0.0)
    scale = torch.maximum(old, need)
    held = codes[flat].view(torch.float8_e4m3fn).float().unflatten(-1, (hkv, d))
    held = held * (old / scale)[:, :, None, :, None]
    new = new[..., None, None]
    was = (pos < past[:, None, None])[..., None, None]
    both = torch.where(new, values / scale[:, :, None, :, None], held).to(torch.float8_e4m3fn).view(torch.uint8)
    both = torch.where(new | was, both, codes[flat].unflatten(-1, (hkv, d))).flatten(-2)
    flat_scales[flat[reached]] = scale[reached]
    codes[flat[reached]] = both[reached]


def _padded(s, x):
    """Packed or batched rows [.., heads, dim] as 32-bit [sequences, longest, heads, dim]."""
    x = x.float()
    if s["uniform"]:
        return x
    out = torch.zeros(s["case"]["seqs"] * s["longest"], *x.shape[2:], device=x.device)
    out[s["slot"]] = x[0]
    return out.unflatten(0, (s["case"]["seqs"], s["longest"]))


def _gathered(s, cache, scales):
    """The cached values of each sequence, [sequences, positions, heads, dim] in 32 bits."""
    table = s["table"].long()
    x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float().unflatten(2, (-1, _BLOCK))
    return x.mul_(scales[table][:, :, :, None, :, None]).flatten(1, 3)


def _plain_attention(s):
    q, c = s["q"], s["case"]
    k, v = _gathered(s, s["k_cache"], s["k_scale"]), _gathered(s, s["v_cache"], s["v_scale"])
    dt, hkv, lead = q.dtype, c["kv_heads"], q.shape[:2]
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


# ---- the definition in 64 bits --------------------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "copy" or work(c)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "paged": _exact_attention}[c["op"]](s, c)


def _exact_rope(s, c):
    rot, out = c["rot"], []
    q_lens, kv_lens = _lengths(c)
    pos = torch.tensor([p for a, b in zip(q_lens, kv_lens) for p in range(b - a, b)], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device="cuda"), torch.outer(pos, s["inv_freq"].double()))
    turn = (turn.conj() if c["backward"] else turn).reshape(-1, 1, rot // 2)
    for x in _q_and_k(s):
        y = x.reshape(-1, x.shape[2], c["dim"]).double().clone()
        if c["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:2], -1, 2).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        out.append(y.reshape(x.shape))
    return tuple(out)


def _round8(x):
    """64-bit x to the nearest 8-bit value, ties to the even one."""
    power = torch.frexp(x)[1].clamp(min=-5) - 4  # of the last place: three bits behind the first, 2^-9 at the least
    return (x * _two_to(-power)).round() * _two_to(power)


def _two_to(power):
    return ((power.long() + 1023) << 52).view(torch.float64)


def _exact_append(s, c):
    q_lens, kv_lens = _lengths(c)
    page, hkv, d = c["page"], c["kv_heads"], c["dim"]
    out, scales_out = [], []
    for name in ("k", "v"):
        cache, scales = s[name + "_cache"].double(), s[name + "_scale"].double()
        x, at = s[name].double().reshape(-1, hkv, d), 0
        for i, (a, b) in enumerate(zip(q_lens, kv_lens)):
            past, lo = b - a, (b - a) // _BLOCK * _BLOCK
            n = -(-b // _BLOCK) - lo // _BLOCK  # blocks of this sequence that change; a ragged edge is laid out as zeros
            rows = torch.zeros(n * _BLOCK, hkv, d, dtype=torch.float64, device=x.device)
            rows[past - lo:past - lo + a] = x[at:at + a]
            at += a
            top = rows.view(n, _BLOCK, hkv, d).abs().amax((1, 3))
            part, power = torch.frexp(top)  # top <= 448 2^e, and 448 = 0.875 2^9
            scale = torch.where(top > 0, _two_to(torch.where(part > 0.875, power - 8, power - 9).clamp(-117, 120)), 2.0 ** -117)
            pos = torch.arange(lo, lo + n * _BLOCK, _BLOCK, device=x.device)
            pages, inside = s["table"][i].long()[pos // page], pos % page // _BLOCK
            if past > lo:
                scale[0] = torch.maximum(scale[0], scales[pages[0], inside[0]])
                first = int(inside[0]) * _BLOCK
                held = cache[pages[0], first:first + past - lo]
                rows[:past - lo] = held * scales[pages[0], inside[0]][:, None]
            scales[pages, inside] = scale
            rows = _round8(rows / scale.repeat_interleave(_BLOCK, 0)[:, :, None])[:b - lo]
            pos = torch.arange(lo, b, device=x.device)
            cache[s["table"][i].long()[pos // page], pos % page] = rows
        out.append(cache)
        scales_out.append(scales)
    return (*out, *scales_out)


def _exact_attention(s, c):
    q_lens, kv_lens = _lengths(c)
    page, hkv, d = c["page"], c["kv_heads"], c["dim"]
    h, group, lead = c["heads"], c["heads"] // hkv, s["q"].shape[:2]
    q = s["q"].reshape(-1, h, d)
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    at = 0
    for i, (a, b) in enumerate(zip(q_lens, kv_lens)):
        rows = s["table"][i, :-(-b // page)].long()
        ki, vi = (s[x + "_cache"].view(torch.uint8)[rows].view(torch.float8_e4m3fn).reshape(-1, hkv, d)[:b].double()
                  * s[x + "_scale"][rows].double().reshape(-1, hkv).repeat_interleave(_BLOCK, 0)[:b, :, None] for x in "kv")
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
