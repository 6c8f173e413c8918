"""A small stack as the operators are used together: a paged-cache layer with rotation, a gated-delta-rule layer and a
hybrid sparse + linear layer on one residual stream, prompts of different lengths and then tokens one by one (the first two
layers' step captured once and replayed).  Every layer's inputs of every step go through the fp64 oracles too."""

import math

import numpy as np
import pytest

import oracle as O
from oracle import delta as OD
from oracle import paged as OP

pytestmark = pytest.mark.gpu

B, DIM, HQ, HKV, D, PAGE, STEPS = 2, 96, 4, 2, 64, 16, 12


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_stack(kind):
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    gen = torch.Generator("cuda").manual_seed(3)
    dev = torch.device("cuda")
    prompts = [70, 37]
    most = max(prompts) + STEPS
    code = torch.float8_e4m3fn if kind == "e4m3" else torch.int8

    def weight(n, m):
        return (torch.randn(n, m, generator=gen, device=dev) / math.sqrt(n)).bfloat16()

    w = {"paged": weight(DIM, (HQ + 2 * HKV) * D), "paged_out": weight(HQ * D, DIM), "delta": weight(DIM, (2 * HKV + HQ) * D),
         "gates": weight(DIM, 2 * HQ), "delta_out": weight(HQ * D, DIM)}
    angle = torch.arange(most, device=dev)[:, None] * 1000.0 ** (-torch.arange(D // 2, device=dev) / (D // 2))
    rope = torch.cat([angle.cos(), angle.sin()], 1).float()
    pages = -(-most // PAGE)
    cache = H.PagedKVCache(B * pages + 2, PAGE, HKV, D, code)
    table = torch.randperm(B * pages + 2, generator=gen, device=dev)[:B * pages].view(B, pages).int()
    states = H.GatedDeltaState(B + 1, HKV, HQ, D, D)
    slots = torch.tensor([2, 0], dtype=torch.int32, device=dev)
    log = []

    def layers(x, cu, lens, max_new, max_len):
        """The first two layers; returns the stream and what each operator was given and gave."""
        qkv = (x @ w["paged"]).view(len(x), -1, D)
        q = cache.append(qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], cu, lens, table, max_new=max_new, rope=rope, q=qkv[:, :HQ])
        a = cache.attend(q, cu, lens, table, max_new=max_new, max_len=max_len)
        y = x + a.flatten(1) @ w["paged_out"]
        qkv2 = (y @ w["delta"]).view(len(x), -1, D)
        qk = torch.nn.functional.normalize(qkv2[:, :2 * HKV].float(), dim=-1).bfloat16()
        gates = (y @ w["gates"]).float()
        g, beta = -torch.nn.functional.softplus(gates[:, :HQ]), torch.sigmoid(gates[:, HQ:]).contiguous()
        o = states.run(qk[:, :HKV], qk[:, HKV:], qkv2[:, 2 * HKV:], g, beta, cu, max_new=max_new, slots=slots)
        return y + o.flatten(1) @ w["delta_out"], (qkv, q, a, qk, qkv2, g, beta, o)

    def keep(got, cu, lens):
        log.append([t.clone() for t in got] + [cu.tolist(), lens.tolist()])

    # prompts
    cu = torch.tensor([0, prompts[0], sum(prompts)], dtype=torch.int32, device=dev)
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    x = torch.randn(sum(prompts), DIM, generator=gen, device=dev).bfloat16()
    y, got = layers(x, cu, lens, max(prompts), max(prompts))
    keep(got, cu, lens)
    # the hybrid layer takes the last token of each prompt and what follows, its own history random
    S, W, Bk, k, T0 = 2, 8, 4, 3, 50
    cfg = H.make_config(B, HQ, HKV, D, Bk, S, W, k, T0 + STEPS)
    hyb = H.HybridAttentionLayer(cfg, dev)
    hyb.k_cache[:, :, :T0] = torch.randn(B, HKV, T0, D, generator=gen, device=dev).bfloat16()
    hyb.v_cache[:, :, :T0] = torch.randn(B, HKV, T0, D, generator=gen, device=dev).bfloat16()
    hyb.init(T0)
    wh = weight(DIM, (HQ + 2 * HKV) * D)

    # tokens: the first two layers' step is captured (one warm step before, on copies of what it changes)
    tok = torch.randn(B, DIM, generator=gen, device=dev).bfloat16()
    cu1 = torch.arange(B + 1, dtype=torch.int32, device=dev)
    saved = [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8), cache.k_scales, cache.v_scales,
                                 states.state)]
    lens += 1
    layers(tok, cu1, lens, 1, most)
    torch.cuda.synchronize()
    for t, s in zip((cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8), cache.k_scales, cache.v_scales, states.state),
                    saved):
        t.copy_(s)
    lens -= 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        y1, got1 = layers(tok, cu1, lens, 1, most)
    hyb_log = []
    for step in range(STEPS):
        graph.replay()
        keep(got1, cu1, lens)
        z = (y1 @ wh).view(B, -1, D)
        args = [t.contiguous() for t in (z[:, :HQ], z[:, HQ:HQ + HKV], z[:, HQ + HKV:])]
        o = hyb.decode_append(*args)
        hyb_log.append((args[0].clone(), o.clone(), hyb.T - 1))
        tok.copy_(torch.nn.functional.normalize(y1.float() + o.flatten(1)[:, :DIM], dim=-1).mul(math.sqrt(DIM)).bfloat16())
    torch.cuda.synchronize()
    assert cache.status() == 0 and states.status() == 0 and hyb.status() == 0 and lens.tolist() == [p + STEPS for p in prompts]

    # the paged layer
    codes = {x: np.zeros((cache.n_pages, HKV, PAGE, D), np.uint8) for x in "kv"}
    scales = {x: np.zeros((cache.n_pages, HKV), np.float32) for x in "kv"}
    tab, ang = table.cpu().numpy(), rope.cpu().numpy()
    S64 = np.zeros((B, HQ, D, D))
    for qkv, q, a, qk, qkv2, g, beta, o, cus, ls in log:
        qkv, q, a, qk, qkv2, g, beta, o = (f64(t) for t in (qkv, q, a, qk, qkv2, g, beta, o))
        for b in range(B):
            r, n, L = slice(cus[b], cus[b + 1]), cus[b + 1] - cus[b], ls[b]
            at = np.arange(L - n, L)
            kk = OP.rotate(qkv[r, HQ:HQ + HKV], ang, at, False).astype(np.float32)
            OP.append(codes["k"], scales["k"], kk, L - n, tab[b], kind, PAGE)
            OP.append(codes["v"], scales["v"], qkv[r, HQ + HKV:].astype(np.float32), L - n, tab[b], kind, PAGE)
            rq = OP.rotate(qkv[r, :HQ], ang, at, False)
            assert (np.abs(q[r] - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -20 * np.abs(rq).max()).all()
            vals = {x: np.concatenate([OP.values(codes[x][p], kind) * scales[x][p].astype(np.float64)[:, None, None]
                                       for p in tab[b]], 1).transpose(1, 0, 2)[:L] for x in "kv"}
            ref, _, mag, _ = OP.attend(q[r], vals["k"], vals["v"], n, L, 1 / math.sqrt(D))
            # a bf16 rounding, one of each weight to 11 bits, and sums in 32 bits
            assert (np.abs(a[r] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag).all()
            kr, qr = qk[r, HKV:], qk[r, :HKV]
            ref, S64[b], mag = OD.run(S64[b], qr, kr, qkv2[r, 2 * HKV:], g[r], beta[r], 1 / math.sqrt(D))
            room = 3 * 2.0 ** -11 * (mag + np.abs(qkv2[r, 2 * HKV:]).max() / math.sqrt(D))
            assert (np.abs(o[r] - ref) <= 2.0 ** -8 * np.abs(ref) + room).all()
    for x, (c, s) in {"k": (cache.k_pages, cache.k_scales), "v": (cache.v_pages, cache.v_scales)}.items():
        used = sorted(set(tab[b, i] for b in range(B) for i in range(-(-(prompts[b] + STEPS) // PAGE))))
        assert np.array_equal(c.view(torch.uint8).cpu().numpy()[used], codes[x][used]) and np.array_equal(s.cpu().numpy()[used], scales[x][used])
    got = f64(states.state)[[2, 0]]
    assert np.linalg.norm(got - S64) <= 8 * math.sqrt(most * D) * 2.0 ** -24 * math.sqrt(most) * np.linalg.norm(S64)
    assert not f64(states.state)[1].any()
    # the hybrid layer, at the parity bars of its own tests
    K, V = f64(hyb.k_cache), f64(hyb.v_cache)
    for q, o, T in hyb_log:
        part = O.partition(T, S, W, Bk)
        q, o = f64(q), f64(o)
        for b in range(B):
            for h in range(HKV):
                rows = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
                mu, var = O.block_stats(K[b, h, :T], part)
                sel = O.select_blocks(O.block_scores(q[b, rows], mu, var, 1 / math.sqrt(D)), k)
                ref = O.hybrid_subtract(q[b, rows], K[b, h, :T], V[b, h, :T], part, sel, 1 / math.sqrt(D))
                assert np.abs(o[b, rows] - ref).max() <= 2e-3


def test_two_streams_at_once():
    """Prompts, single tokens and appends of handles of their own on two streams at once give what they give alone."""
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    gen = torch.Generator("cuda").manual_seed(8)
    lens, news = [700, 333], [[200, 333], [1, 1]]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def make(d):
        table = torch.arange(2 * 11, device="cuda").view(2, 11).int()
        steps = []
        for new in news:
            n = sum(new)
            k = torch.nn.functional.normalize(rand(n, 2, d), dim=-1).bfloat16()
            steps.append((ints([0, new[0], n]), max(new), rand(n, 16, d).bfloat16(), k, rand(n, 2, d).bfloat16(), -0.1 * rand(n, 2).abs(),
                          torch.rand(n, 2, generator=gen, device="cuda")))
        first = torch.randint(-127, 128, (22, 2, 64, d), generator=gen, device="cuda", dtype=torch.int8)
        return table, ints(lens), first, steps

    def run(made, stream=None):
        table, held, first, steps = made
        scale = torch.full(first.shape[:2], 0.01, device="cuda")
        cache = H.PagedKVCache.from_tensors(first.clone(), first.clone(), scale, scale.clone())
        states = H.GatedDeltaState(2, 2, 2, first.shape[3], first.shape[3])
        torch.cuda.synchronize()
        outs = []
        for cu, most, q, k, v, g, beta in steps:
            for _ in range(4):
                cache.append(k, v, cu, held, table, max_new=most, stream=stream)
                outs.append(cache.attend(q, cu, held, table, max_new=most, max_len=max(lens), stream=stream))
                outs.append(states.run(q[:, :2], k, v, g, beta, cu, max_new=most, stream=stream))
        return outs + [cache.k_pages, cache.v_pages, states.state], (cache, states)

    made = [make(64), make(128)]
    alone = [run(m)[0] for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        both = [run(m, s) for m, s in zip(made, streams)]
        torch.cuda.synchronize()
        for (got, handles), want in zip(both, alone):
            assert all(h.status() == 0 for h in handles)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
