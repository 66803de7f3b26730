"""Plain 64-bit forms of the logit constraints (include/gsample.h, "Logit
constraints") and input builders for their tests. Nothing here calls the
library."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # binary32: a rounding is off by at most half a step
# relative half step and smallest subnormal of each output type
HALF_STEP = {0: 2.0 ** -24, 1: 2.0 ** -8, 2: 2.0 ** -11}
TINY = {0: 2.0 ** -149, 1: 2.0 ** -133, 2: 2.0 ** -24}


def clean(rep, freq, pres):
    """The parameters in effect: rep 1 unless finite and > 0, NaN freq/pres 0."""
    rep, freq, pres = (np.asarray(v, np.float32).astype(np.float64) for v in (rep, freq, pres))
    rep = np.where(np.isfinite(rep) & (rep > 0), rep, 1.0)
    return rep, np.where(np.isnan(freq), 0.0, freq), np.where(np.isnan(pres), 0.0, pres)


def constrained(x, history, bias, rep, freq, pres, allowed):
    """Constrained logits in float64 and a bound on the error of the binary32
    evaluation. x, bias: [B, V]; history: uint32 [B, V] words; rep, freq, pres:
    [B]; allowed: bool [B, V].

    The bound: each of the five operations rounds its own result by at most
    U32 of it, and carries the error of its operands (the scaling by rep or
    1 / rep multiplies it); the factor 1.0001 covers the second-order terms and
    the bound's own evaluation."""
    x = np.asarray(x, np.float64)
    rep, freq, pres = (v[:, None] for v in clean(rep, freq, pres))
    h = np.asarray(history, np.uint32)
    c = (h & np.uint32(0x7FFFFFFF)).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        y = x + np.asarray(bias, np.float64)
        e = U32 * np.abs(y)
        seen = h != 0
        k = np.where(y > 0, 1.0 / rep, rep)
        z = np.where(y > 0, y / rep, y * rep)
        e = np.where(seen, e * k + U32 * np.abs(z), e)
        y = np.where(seen, z, y)
        # c is exact up to 2^24; above, its conversion rounds too
        fc = freq * c
        a = y - fc
        r = a - pres
        ea = e + 2 * U32 * np.abs(fc) + U32 * np.abs(a)
        e = np.where(c > 0, ea + U32 * np.abs(r), e)
        y = np.where(c > 0, r, y)
        y = np.where(x == -np.inf, -np.inf, y)
        e = np.where(x == -np.inf, 0.0, e)
    y = np.where(allowed, y, -np.inf)
    e = np.where(allowed, e, 0.0)
    return y, e * 1.0001


def check_values(got, want, err, dtype, where=""):
    """got (float32 array of values of type code `dtype`) against the 64-bit
    values: equal where not finite, else within the evaluation's error plus
    half a step of the output type."""
    got = np.asarray(got, np.float64)
    limit = {0: 3.4028235e38, 1: 3.3895e38, 2: 65504.0}[dtype]
    with np.errstate(invalid="ignore", over="ignore"):
        tol = err + HALF_STEP[dtype] * (np.abs(want) + err) + TINY[dtype]
        ok = np.abs(got - want) <= tol
    special = ~np.isfinite(want)
    ok = np.where(special, (got == want) | (np.isnan(got) & np.isnan(want)), ok)
    # a finite value that rounds past the type's largest may become infinite
    ok |= np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + err >= limit)
    bad = np.argwhere(~ok)
    assert bad.size == 0, "%s: %d values off, first %s: got %r want %r tol %r" % (
        where, len(bad), bad[0], got[tuple(bad[0])], want[tuple(bad[0])], tol[tuple(bad[0])])


def binary32(x, history, bias, rep, freq, pres, allowed):
    """The same formula with every operation rounded once to binary32 (numpy
    float32), for the oracle of the draw."""
    f = np.float32
    x = np.asarray(x, f)
    rep, freq, pres = (v.astype(f)[:, None] for v in clean(rep, freq, pres))
    h = np.asarray(history, np.uint32)
    c = (h & np.uint32(0x7FFFFFFF)).astype(f)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        y = x + np.asarray(bias, f)
        y = np.where(h != 0, np.where(y > 0, y / rep, y * rep), y)
        y = np.where(c > 0, (y - freq * c) - pres, y)
    y = np.where(x == -np.inf, f(-np.inf), y)
    return np.where(allowed, y, f(-np.inf)).astype(f)


def pack_bits(bits):
    """bool [n, V] -> uint32 words [n, ceil(V / 32)], lowest bit first."""
    n, V = bits.shape
    pad = (-V) % 32
    b = np.pad(bits, ((0, 0), (0, pad)))
    return np.packbits(b, axis=1, bitorder="little").view("<u4").reshape(n, -1)


class HostState:
    """The state's arrays on the host, with its three writers in plain form."""

    def __init__(self, rows, vocab, ld=None):
        self.vocab, self.rows = vocab, rows
        self.ld = ld or (vocab + 31) // 32 * 32
        self.history = np.zeros((rows, self.ld), np.uint32)
        self.bias = np.zeros((rows, self.ld), np.float32)
        self.touched = np.zeros((rows, self.ld), bool)

    def append(self, slot, tokens, prompt):
        if not 0 <= slot < self.rows:
            return
        for t in tokens:
            if 0 <= t < self.vocab:
                if prompt:
                    self.history[slot, t] |= np.uint32(0x80000000)
                else:
                    self.history[slot, t] += np.uint32(1)
                self.touched[slot, t] = True

    def set_bias(self, slot, tokens, values):
        if not 0 <= slot < self.rows:
            return
        for t, v in zip(tokens, values):
            if 0 <= t < self.vocab:
                self.bias[slot, t] = v
                self.touched[slot, t] = True

    def reset(self, slot):
        if 0 <= slot < self.rows:
            self.history[slot] = 0
            self.bias[slot] = 0
            self.touched[slot] = False

    def words(self):
        return pack_bits(self.touched)


def random_state(rng, rows, vocab, tokens=40, biases=6, ld=None):
    """A state whose tokens crowd at low ids, so that units hold several
    touched elements, with some biases that ban or force."""
    s = HostState(rows, vocab, ld)
    for r in range(rows):
        ids = np.minimum((vocab ** rng.random(tokens)).astype(np.int64) - 1, vocab - 1)
        cut = tokens // 3
        s.append(r, ids[:cut], True)
        s.append(r, ids[cut:], False)
        s.append(r, [vocab - 1], False)
        b = rng.integers(0, vocab, biases)
        s.set_bias(r, b, rng.uniform(-8, 8, biases).astype(np.float32))
    return s


def random_mask(rng, n, V, kinds=("free", "few", "none", "all", "half")):
    """One mask row per kind in turn: nearly all, a few, no, every, half of the
    tokens allowed."""
    m = np.zeros((n, V), bool)
    for i in range(n):
        k = kinds[i % len(kinds)]
        if k == "free":
            m[i] = rng.random(V) < 0.97
        elif k == "few":
            m[i, rng.integers(0, V, 3)] = True
        elif k == "all":
            m[i] = True
        elif k == "half":
            m[i] = rng.random(V) < 0.5
    return m
