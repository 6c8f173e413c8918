"""The gated delta rule on the GPU against the fp64 oracle.

Tolerances.  State: each token adds rounding errors of 32-bit dot products of dk terms (random in sign, sqrt(dk) 2^-24
of their size), the rule contracts them, so after n tokens the norm of a head's error is within 8 sqrt(n dk) 2^-24 of
the size that went in, |S0| + sqrt(n) |k| max |v| (the 8 covers a few roundings a term and sums of the chunks' 22-bit
operands).  Outputs: half a bf16 step of the value, and single f16 parts of state, update and P in the chunks: 2^-11 each of
sums |S| |q| scale, three of them and the state's error.
"""

import math

import numpy as np
import pytest

from oracle import delta as OD

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


class Delta:
    def __init__(self, new, Hk=2, Hv=4, dk=64, dv=64, slots=None, n_slots=None, seed=0, size=1.0, forget=0.05, tail=0, wide=0, keys=1.0):
        import torch
        import hybrid_sparse_linear_decode_b200 as H
        rng = np.random.default_rng(seed)
        self.torch, self.new = torch, list(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        n = int(self.cu[-1]) + tail
        B = len(new)
        n_slots = n_slots or B

        def rows(heads, d, unit):
            x = rng.standard_normal((n, heads + wide, d))
            x = x / np.linalg.norm(x, axis=-1, keepdims=True) if unit else x * size
            return torch.from_numpy(x).cuda().bfloat16()[:, wide // 2:wide // 2 + heads]

        self.q, self.k, self.v = rows(Hk, dk, True), rows(Hk, dk, True) * keys, rows(Hv, dv, False)
        self.g = torch.from_numpy(-forget * rng.exponential(size=(n, Hv)) * rng.uniform(0, 4, (1, Hv))).float().cuda()
        self.beta = torch.from_numpy(rng.uniform(0, 1, (n, Hv))).float().cuda()
        self.state = torch.from_numpy(rng.standard_normal((n_slots, Hv, dk, dv)) * size).float().cuda()
        self.slots = slots
        self.h = H.GatedDeltaState.from_tensor(self.state, n_k_heads=Hk)
        self.dk, self.dv, self.Hv, self.size, self.keys = dk, dv, Hv, size, keys

    def ints(self, x):
        return self.torch.tensor(np.asarray(x, np.int32), device="cuda")

    def check(self, scale=0.0, max_new=None):
        torch = self.torch
        S0 = f64(self.state)
        n = self.q.shape[0]
        out = torch.full((n, self.Hv, self.dv), 3.0, dtype=torch.bfloat16, device="cuda")
        self.h.run(self.q, self.k, self.v, self.g, self.beta, self.ints(self.cu), max_new=max_new or max(self.new),
                   slots=None if self.slots is None else self.ints(self.slots), scale=scale, out=out)
        assert (out[int(self.cu[-1]):] == 3).all()
        got, S1 = f64(out), f64(self.state)
        want = S0.copy()
        sc = scale or 1 / math.sqrt(self.dk)
        for b, m in enumerate(self.new):
            s = b if self.slots is None else self.slots[b]
            r = slice(self.cu[b], self.cu[b] + m)
            if s < 0 or s >= S0.shape[0]:
                assert (out[r] == 3).all()
                continue
            q, k, v, g, beta = (f64(x[r]) for x in (self.q, self.k, self.v, self.g, self.beta))
            ref, want[s], mag = OD.run(S0[s], q, k, v, g, beta, sc)
            if not m:
                continue
            rel = 8 * math.sqrt(m * self.dk) * 2.0 ** -24
            top = self.keys * np.abs(v).max()
            inn = np.linalg.norm(S0[s], axis=(1, 2)) + math.sqrt(m) * top * math.sqrt(self.dv)
            err = np.linalg.norm(S1[s] - want[s], axis=(1, 2))
            assert (err <= rel * inn).all(), (b, float((err / (rel * inn)).max()))
            room = 3 * 2.0 ** -11 * (mag + sc * top) + (rel * inn * sc)[None, :, None]
            assert (np.abs(got[r] - ref) <= 2.0 ** -8 * np.abs(ref) + room).all(), \
                (b, float((np.abs(got[r] - ref) / (2.0 ** -8 * np.abs(ref) + room)).max()))
        others = [s for s in range(S0.shape[0]) if s not in (range(len(self.new)) if self.slots is None else self.slots)]
        assert np.array_equal(S1[others], S0[others])
        return out


DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("new", [[1], [1, 1, 1], [3, 0, 1, 7], [23, 2], [24], [64, 65, 1], [130, 63, 200, 0], [300]])
def test_delta(dk, dv, new):
    Delta(new, 2, 4, dk, dv, seed=sum(new) + dk, tail=3).check()


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 3), (3, 3), (2, 8)])
@pytest.mark.parametrize("new", [[2, 1], [70, 100]])
def test_delta_heads_and_strides(Hk, Hv, new):
    d = Delta(new, Hk, Hv, 64, 128, seed=Hv, wide=2)
    d.check(scale=0.7)
    assert d.h.status() == 0


@pytest.mark.parametrize("new", [[2, 1, 3, 1], [70, 40, 90, 64]])
def test_delta_slots(new):
    """States in any order; -1 skips a sequence, another index outside too, and is noted."""
    import hybrid_sparse_linear_decode_b200 as H
    d = Delta(new, 1, 2, 64, 64, slots=[5, -1, 0, 3], n_slots=7, seed=1)
    d.check()
    assert d.h.status() == 0
    for bad in (7, -2, 1 << 30):
        d = Delta(new, 1, 2, 64, 64, slots=[5, bad, 0, 3], n_slots=7, seed=2)
        d.check()
        assert d.h.status(clear=True) == H.HYB_STATUS_BAD_SLOT and d.h.status() == 0


@pytest.mark.parametrize("new", [[5, 4], [100, 130]])
@pytest.mark.parametrize("size", [1e-12, 1e-4, 3e4, 1e15])
def test_delta_sizes_of_values(new, size):
    Delta(new, 1, 2, 128, 64, seed=3, size=size).check()


@pytest.mark.parametrize("new", [[5, 4], [13], [14], [100, 130]])
@pytest.mark.parametrize("size", [1e-20, 1e-28, 1e-33])
def test_delta_small_states(new, size):
    """Values far below 1, tokens one by one and in chunks: with values of their size, and read and rewritten with none."""
    Delta(new, 1, 2, 128, 64, seed=3, size=size).check()
    d = Delta(new, 1, 2, 64, 128, seed=13, size=size)
    d.v.zero_()
    d.check()
    d.beta.zero_()
    d.check()


@pytest.mark.parametrize("new", [[13], [14], [150]])
def test_delta_columns_of_different_sizes(new):
    """With no values a state's columns do not meet: each keeps its own precision, whatever its size."""
    d = Delta(new, 1, 2, 128, 128, seed=14)
    d.v.zero_()
    size = 10.0 ** -np.linspace(-20, 33, 128)
    d.state *= d.torch.from_numpy(size).cuda().float()
    S0, (q, k, v, g, beta) = f64(d.state), (f64(x) for x in (d.q, d.k, d.v, d.g, d.beta))
    out = f64(d.h.run(d.q, d.k, d.v, d.g, d.beta, d.ints(d.cu), max_new=max(new)))
    ref, want, mag = OD.run(S0[0], q, k, v, g, beta, 1 / math.sqrt(128))
    rel = 8 * math.sqrt(new[0] * 128) * 2.0 ** -24
    inn = np.linalg.norm(S0[0], axis=1)
    assert (np.linalg.norm(f64(d.state)[0] - want, axis=1) <= rel * inn).all()
    assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * mag + rel * inn / math.sqrt(128)).all()


@pytest.mark.parametrize("new", [[13], [14], [150]])
@pytest.mark.parametrize("size,values", [(1e-30, 1.0), (1e-30, 1e15), (1e-12, 1e18), (1e-37, 1e-30), (0.0, 1e33), (1e20, 1e33),
                                         (0.0, 1e-33)])
def test_delta_values_far_above_the_state(new, size, values):
    d = Delta(new, 1, 2, 64, 64, seed=15, size=values)
    d.state *= size / values
    d.check()


@pytest.mark.parametrize("new", [[5, 4], [64], [100, 130]])
@pytest.mark.parametrize("keys", [2.0 ** -8, 2.0 ** -14, 2.0 ** -30])
def test_delta_short_keys(new, keys):
    """Keys far from length 1, into an empty state: what they leave there is held as finely."""
    d = Delta(new, 1, 2, 128, 128, seed=4, keys=keys)
    d.state.zero_()
    d.check()


@pytest.mark.parametrize("new", [[6], [150]])
def test_delta_decays(new):
    """No decay, strong ones, tokens that forget everything (-inf), long runs of both."""
    for seed, forget in ((1, 0.0), (2, 1.0), (3, 30.0)):
        d = Delta(new, 1, 3, 64, 64, seed=seed, forget=forget)
        d.check()
    d = Delta(new, 1, 3, 64, 64, seed=4)
    d.g[2, 0] = float("-inf")
    d.g[new[0] - 1, 1] = float("-inf")
    d.g[::3, 2] = float("-inf")
    d.check()


@pytest.mark.parametrize("new", [[6], [150]])
def test_delta_learning_rates(new):
    """beta = 0 (nothing written), tiny and one; from an empty state; keys of other sizes with beta |k|^2 < 2."""
    for value in (0.0, 1e-7, 1.0):
        d = Delta(new, 1, 2, 64, 128, seed=5)
        d.beta.fill_(value)
        d.check()
        d = Delta(new, 1, 2, 64, 128, seed=6)
        d.state.zero_()
        d.beta.fill_(value)
        d.check()
    d = Delta(new, 1, 2, 64, 64, seed=7)
    d.k *= 8
    d.beta /= 64
    d.q *= 50
    d.check(scale=0.01)
    d = Delta(new, 1, 2, 64, 64, seed=8)
    d.k[::2] *= 2.0 ** -20
    d.k[:, :, 5] = 0
    d.check()


def test_delta_repeated_keys():
    """The same key again and again: the triangular system is as full as it gets."""
    d = Delta([200], 1, 2, 128, 128, seed=9, forget=0.0)
    d.k[:] = d.k[:1]
    d.beta.fill_(1.0)
    d.check()


def test_steps_continue_what_chunks_began():
    """A prompt in chunks, tokens one by one, and the whole in one call: the same states within their tolerance."""
    import torch
    n = 150
    a, b = Delta([n], 2, 4, 128, 128, seed=10), Delta([n], 2, 4, 128, 128, seed=10)
    whole = a.h.run(a.q, a.k, a.v, a.g, a.beta, a.ints([0, n]), max_new=n)
    parts = []
    for lo, hi in ((0, 100), (100, 101), (101, 104), (104, n)):
        x = [t[lo:hi] for t in (b.q, b.k, b.v, b.g, b.beta)]
        parts.append(b.h.run(*x, b.ints([0, hi - lo]), max_new=hi - lo))
    rel = 16 * math.sqrt(n * 128) * 2.0 ** -24
    assert float((a.state - b.state).norm() / a.state.norm()) <= rel
    assert float((whole.float() - torch.cat(parts).float()).norm() / whole.float().norm()) <= 2.0 ** -8


@pytest.mark.parametrize("new", [[1, 1], [70, 40]])
def test_delta_captured(new):
    """A captured call replayed: the states move on by one step each time."""
    import torch
    d, e = Delta(new, 1, 2, 64, 64, seed=11), Delta(new, 1, 2, 64, 64, seed=11)
    cu = d.ints(d.cu)
    s = torch.cuda.Stream()
    out = torch.empty_like(d.v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        d.h.run(d.q, d.k, d.v, d.g, d.beta, cu, max_new=max(new), out=out)
    for _ in range(3):
        g.replay()
        ref = e.h.run(e.q, e.k, e.v, e.g, e.beta, cu, max_new=max(new), stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(d.state, e.state)


def test_delta_bad_ranges_and_refusals():
    import hybrid_sparse_linear_decode_b200 as H
    d = Delta([4, 4], 1, 2, 64, 64, seed=12)
    for cu in ([0, 9, 3], [0, -4, 8], [5, 2, 8]):
        d.h.run(d.q, d.k, d.v, d.g, d.beta, d.ints(cu), max_new=4)
        assert d.h.status(clear=True) & H.HYB_STATUS_BAD_LENGTH
    d.h.run(d.q, d.k, d.v, d.g, d.beta, d.ints([0, 4, 8]), max_new=2)
    assert d.h.status(clear=True) == H.HYB_STATUS_BAD_LENGTH
    cu = d.ints(d.cu)
    a = [d.q, d.k, d.v, d.g, d.beta]
    for i, bad in ((0, d.q.half()), (1, d.k[:7]), (2, d.v[:, :1]), (3, d.g.double()), (4, d.beta[:, :1])):
        x = list(a)
        x[i] = bad
        with pytest.raises(ValueError):
            d.h.run(*x, cu, max_new=4)
    for kw in (dict(max_new=0), dict(max_new=4, slots=d.ints([0])), dict(max_new=4, slots=cu.long()[:2])):
        with pytest.raises(ValueError):
            d.h.run(*a, cu, **kw)
    with pytest.raises(H.HybAttnError):
        d.h.run(*a, d.ints([0, 1, 2, 3]), max_new=4)     # more sequences than states
    with pytest.raises(H.HybAttnError):
        d.h.run(*a, cu, max_new=4, scale=-1.0)
