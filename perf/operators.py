"""What is measured of the paged 8-bit cache (append with rotation, attention) and of the gated delta rule.

Three operators, each in its plain form (elementary torch operations) and as the
framework's own call:

* ``append``: new keys and values go into a paged cache of 8-bit codes with one
  scale per page and KV head; keys (and queries) are rotated by their position on
  the way.  A page's scale grows when a new token needs it, and the codes that
  the page holds are then rewritten for the new scale.
* ``attend``: causal softmax attention of the newest tokens over such a cache,
  grouped heads, optionally limited to sink tokens and a sliding window.
* ``delta``: S_t = a_t S_{t-1} + k_t (b_t (v_t - a_t S_{t-1}^T k_t))^T,
  o_t = scale S_t^T q_t with a_t = exp(g_t), from a given state to a new one.

Lengths are ragged: sequence b has ``kv_lens[b]`` tokens once its
``cu[b + 1] - cu[b]`` new ones are counted.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ---- the cases ---------------------------------------------------------------------------------
def _append(name, **kw):
    c = dict(op="append", kind="e4m3", dtype="bf16", page=64, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             rotate_q=True, ragged=True)
    return dict(c, **kw, **({"name": name} if name else {}))


def _attend(name, **kw):
    c = dict(op="attend", kind="e4m3", dtype="bf16", page=64, Hq=32, Hkv=8, d=128, window=0, n_sink=0, ragged=True)
    return dict(c, **kw, **({"name": name} if name else {}))


def _delta(name, **kw):
    c = dict(op="delta", Hk=8, Hv=32, d=128, ragged=True)
    return dict(c, **kw, **({"name": name} if name else {}))


def listed():
    return [
        # one token of each of 8 sequences, every layer of every generated token: latency alone
        _append("append_decode_b8", B=8, new=1, len=32768),
        # a few draft tokens each of a small model's sequences: pages end inside the run, short rotary part
        _append("append_drafts_small", B=5, new=17, len=1023, kind="int8", dtype="fp16", page=16, Hq=4, Hkv=1, d=64,
                rot=32, interleaved=True),
        # a prompt of 32K tokens
        _append("append_prompt_32k", B=1, new=32768, len=32768),
        # one user's next token at a moderate length: latency
        _attend("attend_decode_b1_4k", B=1, new=1, len=4096),
        # a full serving batch at 32K, the default workload's shape
        _attend("attend_decode_b8_32k", B=8, new=1, len=32768, ragged=False),
        # the long-context workload's shape, 8-bit integers, sequences of different lengths
        _attend("attend_decode_b4_128k", B=4, new=1, len=131072, kind="int8"),
        # 8 draft tokens per sequence verified at once
        _attend("attend_verify8_b8_32k", B=8, new=8, len=32768),
        # the last 2047 tokens of a prompt of 10001
        _attend("attend_prompt_2k_of_10k", B=1, new=2047, len=10001),
        # a layer that keeps sinks and a window only
        _attend("attend_window_b16", B=16, new=1, len=32768, window=1024, n_sink=4, kind="int8", dtype="fp16", page=32,
                Hq=16, Hkv=8, d=64),
        # one user's next token
        _delta("delta_step_b1", B=1, new=1),
        # the next tokens of a large serving batch: the states' traffic
        _delta("delta_step_b64", B=64, new=1),
        # three prompts, the longest of 8192 tokens
        _delta("delta_prompt_8k", B=3, new=8192),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "delta"))
    if op == "delta":
        Hk = rng.choice((1, 2, 4, 8, 16))
        Hv = Hk * rng.choice((1, 2, 4))
        d = rng.choice((64, 128))
        new = rng.choice((1, _log(rng, 1, 8), _log(rng, 8, 8192)))
        most = max(1, min(64, 3 * 8192 // new, 64 * 32 * 128 * 128 // (Hv * d * d)))
        return _delta(None, B=_log(rng, 1, most), new=new, Hk=Hk, Hv=Hv, d=d, ragged=rng.random() < 0.7)
    Hkv, G, d = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8)), rng.choice((64, 128))
    c = dict(kind=rng.choice(("e4m3", "int8")), dtype=rng.choice(("bf16", "fp16")), page=rng.choice((16, 32, 64, 128)),
             Hkv=Hkv, Hq=Hkv * G, d=d, ragged=rng.random() < 0.7)
    if op == "append":
        new = rng.choice((1, _log(rng, 1, 16), _log(rng, 16, 8192)))
        B = _log(rng, 1, max(1, min(64, 16384 // new)))
        return _append(None, B=B, new=new, len=new + rng.randrange(0, 16384), rot=rng.choice((d, d // 2)),
                       interleaved=rng.random() < 0.5, rotate_q=rng.random() < 0.5, **c)
    new = rng.choice((1, _log(rng, 1, 16), _log(rng, 16, 2048)))
    length = new + _log(rng, 1, 131072) - 1
    # bytes of the cache, and of the plain form's scores, at most the largest listed case's
    most = min(64, 4 * 131072 * 8 * 128 // (length * Hkv * d), 2047 * 10001 * 32 // (new * length * Hkv * G))
    while most < 1:
        length = max(new, length // 2)
        new = min(new, length)
        most = min(64, 4 * 131072 * 8 * 128 // (length * Hkv * d), 2047 * 10001 * 32 // (new * length * Hkv * G))
        new = new if most >= 1 else max(1, new // 2)
    window = rng.choice((0, 0, 0, _log(rng, 1, 4096)))
    return _attend(None, B=_log(rng, 1, most), new=new, len=length, window=window,
                   n_sink=rng.choice((0, 4, 17)) if window else 0, **c)


def _spread(most, n, least, ragged):
    """n lengths in [least, most], the first the longest."""
    if not ragged:
        return [most] * n
    return [max(least, min(most, round(most * (1.0 - 0.75 * ((i * 0.6180339887) % 1.0))))) for i in range(n)]


def _lengths(c):
    """(new tokens, tokens in all) of each sequence."""
    new = _spread(c["new"], c["B"], 1, c["ragged"])
    if c["op"] == "delta":
        return new, new
    return new, [max(n, x) for n, x in zip(new, _spread(c["len"], c["B"], 1, c["ragged"]))]


def work(c):
    new, lens = _lengths(c)
    n = sum(new)
    d = c["d"]
    if c["op"] == "append":
        kv = n * c["Hkv"] * d * 2 * (2 + 1)
        q = n * c["Hq"] * d * 2 * 2 if c["rotate_q"] else 0
        rotated = c["Hkv"] + (c["Hq"] if c["rotate_q"] else 0)
        return {"bytes": kv + q + n * c["rot"] * 4, "flops": n * (rotated * c["rot"] * 3 + 2 * c["Hkv"] * d * 2)}
    if c["op"] == "attend":
        W, S = c["window"], c["n_sink"]
        read = pairs = 0
        for m, L in zip(new, lens):
            if W:
                seen = sum(min(p + 1, W) + max(0, min(S, p + 1 - W)) for p in range(L - m, L))
                read += min(L, min(L, W + m - 1) + min(S, L))
            else:
                seen = m * (L - m) + m * (m + 1) // 2
                read += L
            pairs += seen
        return {"bytes": read * c["Hkv"] * d * 2 + n * c["Hq"] * (d * 2 * 2 + 4), "flops": pairs * c["Hq"] * d * 4}
    state = c["B"] * c["Hv"] * d * d * 4 * 2
    return {"bytes": state + n * (2 * c["Hk"] * d + 2 * c["Hv"] * d) * 2 + n * c["Hv"] * 8,
            "flops": n * c["Hv"] * d * d * 6}


# ---- inputs ------------------------------------------------------------------------------------
def _scale_for(amax, kind):
    """A page's scale: the smallest power of two that holds amax (e4m3), or amax / 127 (int8)."""
    if kind == "int8":
        return (amax / 127.0).clamp_min(2.0 ** -126)
    m, e = torch.frexp(amax)
    x = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 126)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, x, torch.full_like(x, -126)))


def _codes_of(y, kind):
    y = y.clamp(-QMAX[kind], QMAX[kind])
    return torch.round(y).to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    new, lens = _lengths(c)
    B, n = c["B"], sum(new)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s = {"case": c, "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"), "n": n, "max_new": max(new),
         "max_len": max(lens)}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    if c["op"] == "delta":
        d, Hk, Hv = c["d"], c["Hk"], c["Hv"]
        unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
        s["q"] = unit(normal(n, Hk, d)).to(torch.bfloat16)
        s["k"] = unit(normal(n, Hk, d) + 0.5 * normal(1, Hk, d)).to(torch.bfloat16)
        s["v"] = normal(n, Hv, d).to(torch.bfloat16)
        # decays from nearly none to a tenth a token, heads of different rates; learning rates around a half
        rate = torch.exp(2.0 * normal(1, Hv) - 3.0)
        s["g"] = -rate.clamp_max(16.0) * torch.nn.functional.softplus(normal(n, Hv) - 2.0)
        s["beta"] = torch.sigmoid(normal(n, Hv))
        s["slots"] = torch.randperm(B + 2, generator=g, device="cuda")[:B].to(torch.int32)
        s["state"] = normal(B + 2, Hv, d, d) * 0.5
        if own:
            import hybrid_sparse_linear_decode_b200 as H
            s["handle"] = H.GatedDeltaState.from_tensor(s["state"], n_k_heads=Hk)
        return s

    d, Hkv, P, kind, dtype = c["d"], c["Hkv"], c["page"], c["kind"], DTYPES[c["dtype"]]
    need = [-(-x // P) for x in lens]
    n_pages, mp = sum(need) + 3, max(need)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = [0]
    for x in need:
        first.append(first[-1] + x)
    i = torch.arange(mp, device="cuda")
    at = torch.tensor(first[:-1], device="cuda")[:, None] + i
    s["table"] = torch.where(i < torch.tensor(need, device="cuda")[:, None], order[at.clamp_max(n_pages - 1)],
                             torch.full((), -1, dtype=torch.int32, device="cuda"))
    s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for name in ("k", "v"):  # keys have a few strong channels, heads their own size
        size = torch.exp(0.5 * normal(1, Hkv, 1, 1))
        if name == "k":
            size = size * torch.where(normal(1, Hkv, 1, d) > 2.0, 4.0, 1.0)
        x = normal(n_pages, Hkv, P, d) * size
        scale = _scale_for(x.abs().amax((2, 3)), kind)
        s[name + "_scales"] = scale
        s[name + "_pages"] = _codes_of(x * (1.0 / scale)[:, :, None, None], kind)
        if c["op"] == "append":
            s[name] = (normal(n, Hkv, d) * size[0, :, 0]).to(dtype)
        del x
    s["q"] = normal(n, c["Hq"], d).to(dtype)
    if c["op"] == "append":
        r = c["rot"] // 2
        angle = torch.arange(s["max_len"], device="cuda", dtype=torch.float64)[:, None] \
            * 10000.0 ** (-torch.arange(r, device="cuda", dtype=torch.float64) / r)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    if own:
        import hybrid_sparse_linear_decode_b200 as H
        s["handle"] = H.PagedKVCache.from_tensors(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    return s


# ---- the plain forms ---------------------------------------------------------------------------
def _owner(s):
    """The sequence of each new token, and its place among the sequence's new tokens."""
    t = torch.arange(s["n"], device="cuda")
    seq = (t[:, None] >= s["cu"][1:-1]).sum(1)
    return seq, t - s["cu"][seq]


def _rotate(x, rope, pos, c):
    """Pairs of channels turned by their position's angles; products in 64 bits, so that a code next to a border is the right one."""
    r = c["rot"] // 2
    cos, sin = (y.double()[:, None] for y in (rope[pos, :r], rope[pos, r:]))
    x = x.double()
    a, b = (x[..., 0:2 * r:2], x[..., 1:2 * r:2]) if c["interleaved"] else (x[..., :r], x[..., r:2 * r])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if c["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., 2 * r:]], -1).float()


def _append_plain(s):
    c = s["case"]
    P, kind, Hkv = c["page"], c["kind"], c["Hkv"]
    seq, i = _owner(s)
    start = s["kv_lens"] - (s["cu"][1:] - s["cu"][:-1])
    pos = start[seq] + i
    page, slot = s["table"][seq, pos // P].long(), pos % P
    # the page of each sequence that may hold older tokens, and how many of them
    old_page = torch.gather(s["table"], 1, (start // P).long().clamp_max(s["table"].shape[1] - 1)[:, None])[:, 0]
    older = start % P
    held = torch.zeros(s["k_pages"].shape[0] + 1, dtype=torch.bool, device="cuda")
    held[torch.where(older > 0, old_page.long(), held.numel() - 1)] = True
    held = held[:-1, None]
    at = old_page.clamp_min(0).long()
    keep = (torch.arange(P, device="cuda") < older[:, None])[:, None, :, None]
    out = {}
    for name, x in (("k", _rotate(s["k"], s["rope"], pos, c)), ("v", s["v"].float())):
        codes, scales = s[name + "_pages"], s[name + "_scales"]
        amax = torch.zeros_like(scales).scatter_reduce_(0, page[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)[:, None]
        need = _scale_for(amax, kind)
        grown = torch.where(held, torch.maximum(scales, need), need)
        fresh = torch.where(touched, grown, scales)
        inv = 1.0 / fresh
        ratio = (scales[at] * inv[at])[:, :, None, None]
        had = codes[at].float()
        again = _codes_of(had * ratio, kind)
        moved = keep & (fresh[at] != scales[at])[:, :, None, None]
        bits = codes.view(torch.int8)
        bits[at] = torch.where(moved, again.view(torch.int8), bits[at])
        bits[page, :, slot] = _codes_of(x * inv[page][:, :, None], kind).view(torch.int8)
        scales.copy_(fresh)
        out[name + "_pages"], out[name + "_scales"] = codes, scales
    if c["rotate_q"]:
        out["q"] = _rotate(s["q"], s["rope"], pos, c).to(s["q"].dtype)
    return out


def _held(s, name):
    """The cache's values as the sequences see them: [B, Hkv, pages * page, d]."""
    t = s["table"].clamp_min(0).long()
    x = s[name + "_pages"][t].float() * s[name + "_scales"][t][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend_plain(s):
    c = s["case"]
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    seq, i = _owner(s)
    at = (s["cu"][:-1, None] + torch.arange(s["max_new"], device="cuda")).clamp_max(s["n"] - 1)
    q = s["q"][at].float().view(B, s["max_new"], Hkv, -1, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    K, V = _held(s, "k"), _held(s, "v")
    pos = (s["kv_lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(s["max_new"], device="cuda")
    j = torch.arange(K.shape[2], device="cuda")
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["n_sink"])
    seen = (seen & (j < s["kv_lens"][:, None, None]))[:, None, None]
    p = (q @ K.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).unflatten(2, (-1, s["max_new"]))
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ V).unflatten(2, (-1, s["max_new"])) / total.clamp_min(1e-38)
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, i]
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[seq, i]}


def _delta_plain(s):
    """Chunks of 64 tokens: inside a chunk the rule is a unit triangular system, inverted by products."""
    c = s["case"]
    B, Hk, Hv, d = c["B"], c["Hk"], c["Hv"], c["d"]
    C = min(64, s["max_new"])
    chunks = -(-s["max_new"] // C)
    count = s["cu"][1:] - s["cu"][:-1]
    t = torch.arange(chunks * C, device="cuda")
    live = (t < count[:, None])[..., None]
    at = (s["cu"][:-1, None] + t).clamp_max(s["n"] - 1)
    q, k = (s[x][at].float().repeat_interleave(Hv // Hk, 2).unflatten(1, (chunks, C)).transpose(2, 3) for x in ("q", "k"))
    v = s["v"][at].float().unflatten(1, (chunks, C)).transpose(2, 3)
    g = torch.where(live, s["g"][at].double(), 0.0).unflatten(1, (chunks, C)).transpose(2, 3).cumsum(-1)
    beta = torch.where(live, s["beta"][at], 0.0).unflatten(1, (chunks, C)).transpose(2, 3)[..., None]
    low = torch.ones(C, C, device="cuda").tril()
    # decays from s to t >= s; chunks are in dimension 1, heads in 2
    decay = (g[..., :, None] - g[..., None, :]).masked_fill_(low == 0, -math.inf).exp_().float()
    since, left, whole = g.exp().float()[..., None], (g[..., -1:] - g).exp().float()[..., None], g[..., -1].exp().float()
    A = -(beta * (k @ k.transpose(-1, -2)) * decay).tril(-1)
    T = torch.eye(C, device="cuda") + A
    for _ in range(max(0, (C - 1).bit_length() - 1)):
        A = A @ A
        T = T + T @ A
    scale = 1.0 / math.sqrt(d)
    inner = (q @ k.transpose(-1, -2)) * decay
    state = s["state"][s["slots"].long()]
    out = torch.empty(B, chunks, Hv, C, d, device="cuda")
    for n in range(chunks):
        fresh = T[:, n] @ (beta[:, n] * (v[:, n] - since[:, n] * (k[:, n] @ state)))
        out[:, n] = scale * (since[:, n] * (q[:, n] @ state) + inner[:, n] @ fresh)
        state = whole[:, n, :, None, None] * state + k[:, n].transpose(-1, -2) @ (left[:, n] * fresh)
    s["state"][s["slots"].long()] = state
    seq, i = _owner(s)
    return {"out": out.transpose(2, 3).flatten(1, 2)[seq, i].to(torch.bfloat16), "state": s["state"]}


def run(s):
    c = s["case"]
    if not own:
        return {"append": _append_plain, "attend": _attend_plain, "delta": _delta_plain}[c["op"]](s)
    h = s["handle"]
    if c["op"] == "append":
        q = h.append(s["k"], s["v"], s["cu"], s["kv_lens"], s["table"], max_new=s["max_new"], rope=s["rope"],
                     interleaved=c["interleaved"], q=s["q"] if c["rotate_q"] else None)
        out = {"k_pages": s["k_pages"], "k_scales": s["k_scales"], "v_pages": s["v_pages"], "v_scales": s["v_scales"]}
        return dict(out, q=q) if c["rotate_q"] else out
    if c["op"] == "attend":
        out, lse = h.attend(s["q"], s["cu"], s["kv_lens"], s["table"], max_new=s["max_new"], max_len=s["max_len"],
                            window=c["window"], n_sink=c["n_sink"], return_lse=True)
        return {"out": out, "lse": lse}
    out = h.run(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], slots=s["slots"], max_new=s["max_new"])
    return {"out": out, "state": s["state"]}


# ---- from the definitions, in 64 bits, sequence by sequence ----------------------------------------
def _exact_append(s, c):
    P, kind, r = c["page"], c["kind"], c["rot"] // 2
    new, lens = _lengths(c)
    first, second = (range(0, 2 * r, 2), range(1, 2 * r, 2)) if c["interleaved"] else (range(r), range(r, 2 * r))
    first, second = (torch.tensor(list(x), device="cuda") for x in (first, second))

    def turn(x, at):
        x = x.double()
        y = x.clone()
        w = s["rope"][at].double()[:, None]
        y[..., first] = x[..., first] * w[..., :r] - x[..., second] * w[..., r:]
        y[..., second] = x[..., second] * w[..., :r] + x[..., first] * w[..., r:]
        return y

    def rounded(y):
        y = y.clamp(-QMAX[kind], QMAX[kind])
        if kind == "int8":
            return y.round()
        # e4m3: 4 significant bits, the smallest step 2^-9
        step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 4).clamp_min(-9))
        return (y / step).round() * step

    def fitting(top):
        if kind == "int8":
            return max(top / 127.0, 2.0 ** -126)
        x = -126
        while 448.0 * 2.0 ** x < top:
            x += 1
        return 2.0 ** x

    if sum(new) > 20000:
        return None
    pages = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
    scales = {"k": s["k_scales"].double(), "v": s["v_scales"].double()}
    qs = []
    t = 0
    for b, (m, L) in enumerate(zip(new, lens)):
        at = torch.arange(L - m, L, device="cuda")
        rows = {"k": turn(s["k"][t:t + m], at), "v": s["v"][t:t + m].double()}
        qs.append(turn(s["q"][t:t + m], at))
        t += m
        for lo in range((L - m) // P * P, L, P):
            p = int(s["table"][b, lo // P])
            a, z = max(lo, L - m), min(lo + P, L)
            for name, x in rows.items():
                x = x[a - (L - m):z - (L - m)]
                want = torch.tensor([fitting(float(w)) for w in x.abs().amax((0, 2)).cpu()], dtype=torch.float64, device="cuda")
                was = scales[name][p].clone()
                now = torch.maximum(was, want) if a > lo else want
                if a > lo:
                    grew = (now != was)[:, None, None]
                    had = pages[name][p, :, :a - lo]
                    pages[name][p, :, :a - lo] = torch.where(grew, rounded(had * (was / now)[:, None, None]), had)
                pages[name][p, :, a - lo:z - lo] = rounded(x / now[:, None]).transpose(0, 1)
                scales[name][p] = now
    out = {}
    for name in ("k", "v"):
        out[name + "_pages"] = pages[name] if kind == "e4m3" else None
        out[name + "_scales"] = scales[name]
    return dict(out, q=torch.cat(qs)) if c["rotate_q"] else out


def _exact_attend(s, c):
    new, lens = _lengths(c)
    P, G, d = c["page"], c["Hq"] // c["Hkv"], c["d"]
    out = torch.zeros(s["n"], c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["n"], c["Hq"], dtype=torch.float64, device="cuda")
    t = 0
    for b, (m, L) in enumerate(zip(new, lens)):
        pages = s["table"][b, :-(-L // P)].long()
        pos = torch.arange(L - m, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        hidden = j > pos
        if c["window"]:
            hidden |= (j <= pos - c["window"]) & (j >= c["n_sink"])
        for h in range(c["Hkv"]):
            K, V = ((s[x + "_pages"][pages, h].double() * s[x + "_scales"][pages, h].double()[:, None, None]).flatten(0, 1)[:L]
                    for x in ("k", "v"))
            for u in range(h * G, h * G + G):
                z = s["q"][t:t + m, u].double() @ K.T / math.sqrt(d)
                z = z.masked_fill(hidden, -math.inf)
                lse[t:t + m, u] = torch.logsumexp(z, 1)
                out[t:t + m, u] = torch.exp(z - lse[t:t + m, u][:, None]) @ V
        t += m
    return {"out": out, "lse": lse}


def _exact_delta(s, c):
    new, _ = _lengths(c)
    rep = c["Hv"] // c["Hk"]
    state = s["state"].double()
    S = state[s["slots"].long()]
    out = torch.zeros(s["n"], c["Hv"], c["d"], dtype=torch.float64, device="cuda")
    starts = s["cu"][:-1].long()
    count = torch.tensor(new, device="cuda")
    for i in range(max(new)):
        live = count > i
        row = torch.where(live, starts + i, starts)
        k = s["k"][row].double().repeat_interleave(rep, 1)
        q = s["q"][row].double().repeat_interleave(rep, 1)
        a = torch.where(live[:, None], s["g"][row].double().exp(), 1.0)[..., None, None]
        S = S * a
        miss = s["v"][row].double() - (S * k[..., None]).sum(2)
        S = S + torch.where(live[:, None], s["beta"][row].double(), 0.0)[..., None, None] * k[..., None] * miss[:, :, None]
        got = (S * q[..., None]).sum(2) / math.sqrt(c["d"])
        out[row] = torch.where(live[:, None, None], got, out[row])
    state[s["slots"].long()] = S
    return {"out": out, "state": state}


def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "attend": _exact_attend, "delta": _exact_delta}[c["op"]](s, c)
