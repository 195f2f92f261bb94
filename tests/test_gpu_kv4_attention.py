"""GPU attention over the paged 4-bit cache against the float64 oracle.

Tolerance, from the arithmetic (u = 2^-24), for an output channel with S = sum_t p_t |v_t|, n tokens seen,
A = max_t scale sum_c |q_c k_c|, V = max |v| (test_gpu_attention.py has the terms of the scores, which are the same
products and sums: E = u (42 A + A' + 3 (2 A + 56) + n / 32 + 40)):
  few rows    weights times V scales are rounded once to fp16: 2^-11, and below 2^-14 by 2^-25, where the largest
              product of the row is at least 2^14 (an octave for the power of two that bounds its scale): n 2^-39 of the
              row's largest p v_scale, times a code of 6, in which V is one: n 2^-36 V bounds it
              |out - out64| <= 2^-8 |out64| + S (2^-11 + 2 E) + n 2^-36 V
  many rows   K, V and the weights are rounded to 11 bits each: E grows by 2^-11 A (and by 2^-25 scale sum |q| below
              fp16's normal range, less than A' u for the keys here), the output's error by 2^-11 S; a row's largest
              weight is 2^7 at least: n 2^-31 V
and |lse - lse64| <= 2 E + u |lse|."""
import math

import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle import kvcache, layer
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _gpu(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a)).view(dt).to(dev())


class Problem:
    """A 4-bit cache whose pages hold the sequences' tokens, and NaN and infinite scales everywhere else."""

    def __init__(self, seed, nqs, lens, Hq, Hk, D, page, spare=2, each=True, qgain=1.0, octaves=3):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hk, self.D, self.page, self.lens, self.nqs = Hq, Hk, D, page, list(lens), list(nqs)
        B, self.T = len(lens), sum(nqs)
        need = [-(-L // page) for L in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        table = np.full((B, max(max(need), 1) + 1), 1 << 30, np.int64)         # entries of no token: never read
        table[rng.random(table.shape) < 0.5] = -7
        at = 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.table, self.pool = table, pages * page
        P = self.pool
        kc, vc = (rng.integers(0, 256, size=(P, Hk, D // 2)).astype(np.uint8) for _ in range(2))
        ks, vs = np.full((P, Hk, D // 32), 0x7E00, np.uint16), np.full((P, Hk, D // 32), 0x7C00, np.uint16)
        for b in range(B):
            if lens[b] == 0:
                continue
            s = layer.slots_of(table[b], lens[b], page, P)
            gain = np.repeat(2.0 ** rng.integers(-octaves, octaves + 1, size=(lens[b], Hk, D // 32)), 32, -1)
            k = rng.standard_normal((lens[b], Hk, D)) * (1 + 4 * (rng.random((1, Hk, D)) < 0.05))
            kc[s], ks[s] = kvcache.kv4_quantize_values(k)
            vc[s], vs[s] = kvcache.kv4_quantize_values(rng.standard_normal((lens[b], Hk, D)) * gain)
        self.host = [kc, ks, vc, vs]
        self.upload()
        self.qb = oracle.f32_to_bf16_bits((qgain * rng.standard_normal((self.T, Hq, D))).astype(np.float32))
        self.q = bf16_to_gpu(self.qb)
        self.bt = torch.from_numpy(table.astype(np.int32)).to(dev())
        self.sl = torch.tensor(lens, dtype=torch.int32, device=dev())
        self.starts = np.concatenate([[0], np.cumsum(nqs)])
        self.q0 = None if each and all(n == 1 for n in nqs) else _gpu(self.starts.astype(np.int32), torch.int32)

    def upload(self):
        kc, ks, vc, vs = self.host
        self.cache = qlq.QuantizedKV4(_gpu(kc, torch.uint8), _gpu(ks, torch.float16), _gpu(vc, torch.uint8),
                                      _gpu(vs, torch.float16))

    def used(self, b):
        return layer.slots_of(self.table[b], self.lens[b], self.page, self.pool)

    def values(self):
        kc, ks, vc, vs = self.host
        return kvcache.kv4_values(kc, ks), kvcache.kv4_values(vc, vs)

    def run(self, **kw):
        return qlq.kv_attention(self.q, self.cache, self.bt, self.sl, self.page, q_start=self.q0, **kw)

    def check(self, scale=None, causal=True, window=0, what=""):
        lse = torch.full((self.T, self.Hq), 123.0, device=dev())
        out = self.run(scale=scale, causal=causal, window=window, lse=lse)
        self.compare(out, lse, self.table, self.lens, scale, causal, window, what)
        return out

    def compare(self, out, lse, table, lens, scale=None, causal=True, window=0, what=""):
        q, (k, v) = bits_to_f64(self.qb), self.values()
        sc = self.D ** -0.5 if scale is None else scale
        o64, l64, written, S = layer.kv_attention(q, k, v, table, lens, self.page, self.starts, sc, causal, window)
        used = np.concatenate([layer.slots_of(table[b], lens[b], self.page, self.pool) for b in range(len(lens))]).astype(int)
        used = used[used >= 0]
        ku, vu, n = np.abs(k[used]), np.abs(v[used]), max(lens)
        V = vu.max() if used.size else 0.0
        A1 = abs(sc) * np.abs(q).max() * ku.sum(-1).max() if used.size else 0.0
        A = abs(sc) * max((np.abs(q[:, h]) @ ku[:, h // (self.Hq // self.Hk)].T).max() for h in range(self.Hq)) if used.size else 0.0
        E = U * (42 * A + A1 + 3 * (2 * A + 56) + n / 32 + 40)
        W, tail = 2.0 ** -11, 2.0 ** -36
        if -(-self.T // len(lens)) * (self.Hq // self.Hk) > {32: 96, 64: 96, 256: 256}.get(self.D, 64):
            E, W, tail = E + 2.0 ** -11 * A + U * A1, 2 * W, 2.0 ** -31
        got = bits_to_f64(bf16_bits(out))
        assert np.all(np.isfinite(got)), what
        over = np.abs(got - o64) - (2.0 ** -8 * np.abs(o64) + S * (W + 2 * E) + n * tail * V + 1e-38)
        assert np.max(over) <= 0, f"{what}: {np.max(over):.3e} beyond the bound at {np.unravel_index(over.argmax(), over.shape)}"
        if lse is not None:
            lg, empty = lse.cpu().numpy().astype(np.float64), np.isneginf(l64)
            assert np.array_equal(np.isneginf(lg), empty), what
            if (~empty).any():
                d = np.abs(lg[~empty] - l64[~empty]) - (2 * E + U * np.abs(l64[~empty]))
                assert d.max() <= 0, f"{what}: lse {d.max():.3e} beyond the bound"


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 100, 255, 256, 257, 1000, 2049]


@pytest.mark.parametrize("heads", [(1, 1, 32), (4, 4, 64), (28, 4, 128), (3, 1, 96), (16, 2, 192), (8, 2, 256), (20, 1, 128),
                                   (40, 1, 64), (32, 8, 128), (18, 1, 96)])
@pytest.mark.parametrize("page", [16, 256])
def test_single_tokens_ragged_lengths(heads, page):
    Hq, Hk, D = heads
    print(f"attention4 heads={heads} page={page}", flush=True)
    p = Problem(Hq + D + page, [1] * len(LENS), LENS, Hq, Hk, D, page)
    a = p.check(what="decode")
    p.q0 = _gpu(p.starts.astype(np.int32), torch.int32)               # the same through q_start
    assert a.shape == p.check(what="decode through q_start").shape


# Neighbouring KV heads that a workgroup takes together, by their number and channels: eight, four, two and ones
# that have none, and query rows of one and of two groups of 16.
TOGETHER = [(8, 8, 64), (16, 16, 64), (8, 4, 128), (12, 12, 128), (16, 8, 128), (20, 20, 128), (2, 2, 256), (6, 6, 256),
            (12, 12, 256), (8, 8, 256), (6, 6, 64), (10, 10, 128), (3, 3, 256), (12, 6, 96)]


@pytest.mark.parametrize("heads", TOGETHER)
@pytest.mark.parametrize("page", [16, 64])
def test_neighbouring_heads(heads, page):
    Hq, Hk, D = heads
    print(f"attention4 neighbouring heads={heads} page={page}", flush=True)
    p = Problem(Hq + D + page, [1] * 6, [0, 1, 31, 700, 4099, 12345], Hq, Hk, D, page)
    a = p.check(what="decode")
    assert torch.equal(a, p.run()), "the same again"
    p.check(window=100, what="decode, window")
    p = Problem(Hq + D, [3, 1, 0, 11], [3, 900, 40, 2000], Hq, Hk, D, page, each=False)
    p.check(what="several query tokens")
    p.check(causal=False, what="not causal")
    p.check(window=70, what="several query tokens, window")
    p = Problem(Hq * D, [26], [5000], Hq, Hk, D, page, each=False)       # rows of the second group
    p.check(what="one sequence")


@pytest.mark.parametrize("heads", [(8, 8, 64), (4, 4, 128), (8, 8, 128), (2, 2, 256), (8, 8, 256)])
def test_neighbouring_heads_bad_pages_and_unseen_entries(heads):
    Hq, Hk, D = heads
    print(f"attention4 neighbouring heads, bad pages heads={heads}", flush=True)
    p = Problem(D + Hk, (1, 1, 1), (200, 64, 890), Hq, Hk, D, 16, each=False)
    t = p.table.copy()
    t[0, 2], t[1, :], t[2, 0], t[2, 5], t[0, 7] = -1, p.pool // 16, 1 << 30, -(1 << 31), p.pool // 16
    out, lse = torch.full((p.T, Hq, D), 9.0, dtype=torch.bfloat16, device=dev()), torch.zeros((p.T, Hq), device=dev())
    qlq.kv_attention(p.q, p.cache, _gpu(t.astype(np.int32), torch.int32), p.sl, 16, q_start=p.q0, out=out, lse=lse)
    p.compare(out, lse, t, p.lens, what="bad pages")
    assert not out[1].any()
    out = p.check(window=40, what="before")
    for b, L in enumerate(p.lens):
        at = torch.from_numpy(p.used(b)[:L - 40]).to(dev())
        p.cache.k_codes[at], p.cache.v_codes[at] = 0x77, 0xFF
        p.cache.k_scales[at], p.cache.v_scales[at] = float("nan"), float("inf")
    assert torch.equal(p.run(window=40), out)


@pytest.mark.parametrize("heads", [(64, 64, 32), (48, 48, 64), (96, 24, 96), (10, 10, 192)])
def test_heads_of_long_lines_together(heads):
    # more than ten tiles of 32 tokens for every wave of a head: a workgroup's waves take neighbouring heads; and one
    # token less per sequence, where lengths change the choice under one and the same launch
    Hq, Hk, D = heads
    groups = Hk // (4 if Hk % 4 == 0 else 2)
    waves = max(256 // groups // 8 * 8, 1) * (8 if D <= 128 else 4) * groups // Hk
    n = 32 * (10 * waves // 3 + 4)
    print(f"attention4 long lines heads={heads} tokens=3x{n}", flush=True)
    p = Problem(D, [1, 1, 1], [n + 5, n, n - 700], Hq, Hk, D, 64)
    a = p.check(what="together")
    p.lens = [n // 2, n, 9]
    p.sl.copy_(torch.tensor(p.lens, dtype=torch.int32))
    p.check(what="one head each")
    p.lens = [n + 5, n, n - 700]
    p.sl.copy_(torch.tensor(p.lens, dtype=torch.int32))
    assert torch.equal(p.run(), a)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 4096])
def test_page_sizes(page):
    Problem(page, [1, 1, 1], [5, 33, 300], 4, 2, 64, page).check(what=f"page {page}")


@pytest.mark.parametrize("window", [0, 1, 7, 64, 100000])
@pytest.mark.parametrize("nqs", [(1, 2, 5, 33), (17, 0, 1, 64), (130, 3, 0, 0), (4, 40, 300, 9)])
def test_many_query_tokens(nqs, window):
    lens = [max(n, 1) + e for n, e in zip(nqs, (300, 0, 31, 1000))]
    print(f"attention4 nqs={nqs} lens={lens} window={window}", flush=True)
    for Hq, Hk, D in ((4, 2, 64), (7, 1, 128)):
        Problem(sum(nqs) + window, nqs, lens, Hq, Hk, D, 16, each=False).check(window=window, what=f"{Hq},{Hk},{D}")


@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (5, 1, 96), (3, 1, 32), (2, 1, 256), (6, 3, 192)])
@pytest.mark.parametrize("nqs", [(300, 1, 0, 40), (64, 64), (1000,), (50, 3, 20), (9, 2)])
def test_prompt_chunks(heads, nqs):
    Hq, Hk, D = heads
    lens = [n + e for n, e in zip(nqs, (0, 700, 5, 333))]
    print(f"attention4 prompt chunks heads={heads} nqs={nqs}", flush=True)
    p = Problem(sum(nqs) + D, nqs, lens, Hq, Hk, D, 16 if D % 64 else 64, each=False)
    p.check(what="causal")
    p.check(window=70, what="window")
    if len(nqs) == 2:
        p.check(causal=False, scale=-0.2, what="no mask, negative scale")


def test_no_causal_mask_scale_and_large_scores():
    p = Problem(5, (9, 1), (77, 130), 4, 2, 64, 32, each=False)
    p.check(causal=False, what="no mask")
    p.check(scale=0.0, what="scale 0: a plain mean")
    p.check(scale=-0.3, what="negative scale")
    Problem(6, (1, 1), (900, 40), 4, 2, 64, 32, qgain=2.0 ** 6).check(what="large scores")
    Problem(7, (1, 1), (900, 40), 4, 2, 64, 32, qgain=2.0 ** -40).check(what="tiny queries")


def test_more_queries_than_tokens_leave_rows_empty():
    for seed, nqs, lens in ((8, (5, 40, 3), (2, 0, 3)), (9, (90, 64, 80), (200, 0, 40))):
        p = Problem(seed, nqs, lens, 4, 2, 64, 16, each=False)
        out = p.check(what="nq > L")
        a = nqs[0]
        assert not out[a:a + nqs[1]].any()
        assert not out[:max(0, nqs[0] - lens[0])].any() and not out[a + nqs[1]:a + nqs[1] + max(0, nqs[2] - lens[2])].any()


@pytest.mark.parametrize("nqs", [(2, 1, 3), (90, 40, 70)])
def test_rows_outside_the_sequences_and_lengths_out_of_range(nqs):
    p = Problem(9, nqs, [n + e for n, e in zip(nqs, (38, 19, 77 if nqs[2] == 3 else 74))], 4, 2, 64, 16, each=False)   # the last: whole pages
    T = p.T + 4
    q = torch.zeros((T, 4, 64), dtype=torch.bfloat16, device=dev())
    q[2:2 + p.T] = p.q
    out, lse = torch.full_like(q, 3.0), torch.full((T, 4), 3.0, device=dev())
    qlq.kv_attention(q, p.cache, p.bt, p.sl, 16, q_start=(p.q0 + 2).contiguous(), out=out, lse=lse)
    p.compare(out[2:2 + p.T].contiguous(), lse[2:2 + p.T], p.table, p.lens)
    for t in (out, lse):
        assert bool((t[:2] == 3.0).all()) and bool((t[2 + p.T:] == 3.0).all())
    # a negative length is empty; a length above the table's tokens stops there (its pages there are bad ones)
    sl = torch.tensor([-5, p.lens[1], 1 << 30], dtype=torch.int32, device=dev())
    out2 = qlq.kv_attention(q, p.cache, p.bt, sl, 16, q_start=(p.q0 + 2).contiguous())
    p.compare(out2[2:2 + p.T].contiguous(), None, p.table, [0, p.lens[1], p.table.shape[1] * 16], what="bounded lengths")
    wild = torch.tensor([2, 4, 5, 1 << 30], dtype=torch.int32, device=dev())
    guard = torch.full((T + 64, 4, 64), 3.0, dtype=torch.bfloat16, device=dev())
    qlq.kv_attention(q, p.cache, p.bt, p.sl, 16, q_start=wild, out=guard[:T])
    assert bool((guard[T:] == 3.0).all()) and bool((guard[:2] == 3.0).all())


@pytest.mark.parametrize("nqs", [(1, 1, 4), (90, 64, 80)])
def test_bad_pages_are_left_out(nqs):
    p = Problem(10, nqs, (200, 64, 190), 4, 2, 64, 16, each=False)
    t = p.table.copy()
    t[0, 2], t[1, :], t[2, 0], t[2, 5], t[0, 7] = -1, p.pool // 16, 1 << 30, -(1 << 31), p.pool // 16
    out, lse = torch.full((p.T, 4, 64), 9.0, dtype=torch.bfloat16, device=dev()), torch.zeros((p.T, 4), device=dev())
    qlq.kv_attention(p.q, p.cache, _gpu(t.astype(np.int32), torch.int32), p.sl, 16, q_start=p.q0, out=out, lse=lse)
    p.compare(out, lse, t, p.lens, what="bad pages")
    assert not out[nqs[0]:nqs[0] + nqs[1]].any()


@pytest.mark.parametrize("case", [((1, 1, 1), (700, 1003, 90)), ((3, 1, 9), (700, 1003, 90)), ((150, 64, 80), (850, 1067, 170))])
@pytest.mark.parametrize("window", [1, 40, 333])
def test_entries_that_no_query_sees_may_hold_anything(case, window):
    nqs, lens = case
    print(f"attention4 unseen entries nqs={nqs} window={window}", flush=True)
    for Hq, Hk, D in ((4, 2, 64), (2, 1, 96), (4, 1, 128), (2, 1, 256)):
        p = Problem(sum(nqs) + D + window, nqs, lens, Hq, Hk, D, 16, each=max(nqs) == 1)
        out = p.check(window=window, what="before")
        lse, lse2 = torch.zeros(p.T, Hq, device=dev()), torch.zeros(p.T, Hq, device=dev())
        p.run(window=window, lse=lse)
        for scale in (float("nan"), float("inf")):
            for b, (n, L) in enumerate(zip(nqs, lens)):
                at = torch.from_numpy(p.used(b)[:max(0, L - n - window + 1)]).to(dev())
                p.cache.k_codes[at], p.cache.v_codes[at] = 0x77, 0xFF
                p.cache.k_scales[at], p.cache.v_scales[at] = scale, scale
            assert torch.equal(p.run(window=window, lse=lse2), out) and torch.equal(lse2, lse), (Hq, Hk, D, scale)


@pytest.mark.parametrize("nqs", [(1, 1), (40, 30), (100, 70)])
def test_scales_of_every_size(nqs):
    # K scales up to fp16's largest and V scales over 36 octaves, group by group, within a tile and from tile to tile
    p = Problem(22, nqs, (300, 260), 4, 2, 64, 32, each=False, qgain=2.0 ** -14)
    rng = np.random.default_rng(5)
    for b in range(2):
        s = p.used(b)
        big = s[rng.random(s.size) < 0.02]
        p.host[1][big] = oracle.fp16_encode(np.full(p.host[1][big].shape, 60000.0, np.float32))
        p.host[3][s] = oracle.fp16_encode((2.0 ** rng.uniform(-23, 13, size=p.host[3][s].shape)).astype(np.float32))
    p.upload()
    p.check(what="scales of every size")


@pytest.mark.parametrize("octaves", [12, 20, 24])
@pytest.mark.parametrize("nqs", [(1,), (1, 1, 1, 1), (150,)])
def test_a_quiet_group_beside_a_loud_one(nqs, octaves):
    # every token's second group has V scales `octaves` below the first: each group to its own bound
    for Hq, Hk, D in ((4, 2, 64), (4, 1, 128)):
        p = Problem(octaves, nqs, [600 + n for n in nqs], Hq, Hk, D, 32, each=False, octaves=0)
        for b in range(len(nqs)):
            s = p.used(b)
            p.host[3][s, :, 0] = oracle.fp16_encode(np.full((s.size, Hk), 2.0 ** 6, np.float32))
            p.host[3][s, :, 1] = oracle.fp16_encode(np.full((s.size, Hk), 2.0 ** (6 - octaves) * 1.2, np.float32))
        p.upload()
        out = p.check(what="both")
        o64, _, _, S = layer.kv_attention(bits_to_f64(p.qb), *p.values(), p.table, p.lens, p.page, p.starts)
        g = bits_to_f64(bf16_bits(out))[..., 32:64]
        # the weight times its scale is 2^(15 - 1 - octaves) of the largest or more for every weight that counts: 2^-11
        # down to 2^-28 of it, so below 2^(octaves - 28) of a row's largest weight a token may be off by 2^-25 of the unit
        E = 2.0 ** -9 if max(nqs) > 1 else 2.0 ** -16
        W = 2.0 ** -10 if max(nqs) > 1 else 2.0 ** -11
        tail = 650 * 2.0 ** (octaves - 38 + (6 if max(nqs) > 1 else 0)) * 6 * 2.0 ** (6 - octaves) * 1.2
        over = np.abs(g - o64[..., 32:64]) - (2.0 ** -8 * np.abs(o64[..., 32:64]) + S[..., 32:64] * (W + 2 * E) + tail)
        assert over.max() <= 0, over.max()


@pytest.mark.parametrize("octaves", [20.0, 25.2, 33.0])
@pytest.mark.parametrize("heads", [(4, 1, 64), (4, 4, 128), (8, 2, 96), (2, 1, 192), (2, 1, 256), (3, 1, 32)])
@pytest.mark.parametrize("BL", [(1, 32), (300, 3000)])
def test_tail_far_below_the_largest_weight(BL, heads, octaves):
    # One token outweighs every other by `octaves`, and half of the channels are zero in its values: there the output is
    # the others' alone.  Weights below 2^-28 of the largest are off by 2^-39 of it (all V scales here are one power of two).
    (B, L), (Hq, Hk, D) = BL, heads
    print(f"tail4 B={B} L={L} heads={heads} octaves={octaves}", flush=True)
    rng = np.random.default_rng(L + D)
    page = 32
    pages = -(-L // page)
    P, top = pages * page, L // 3
    k = rng.integers(-6, 7, size=(P, Hk, D)).astype(np.float64)
    k = np.sign(k) * kvcache.E2M1[np.abs(k).astype(int)] * 2.0 ** -4
    k[:, :, 0] = 0
    k[top, :, 0] = 1.0 / 4
    v = kvcache.E2M1[rng.integers(1, 8, size=(P, Hk, D))]
    v[top, :, ::2] = 0
    pack = lambda x, s: kvcache.e2m1_encode(x, s)[..., kvcache.kv4_order(D)]
    kc, vc = pack(k, 2.0 ** -4), pack(v, 1.0)
    both = lambda c: _gpu(c[..., 0::2] | c[..., 1::2] << 4, torch.uint8)
    ks, vs = (torch.full((P, Hk, D // 32), x, dtype=torch.float16, device=dev()) for x in (2.0 ** -4, 1.0))
    q = np.zeros((Hq, D), np.float32)
    q[:, 0] = 4 * octaves * np.log(2.0) * (1 + np.arange(Hq) / 256)
    qb = oracle.f32_to_bf16_bits(q)
    table = torch.arange(pages, dtype=torch.int32, device=dev()).expand(B, pages).contiguous()
    lens = torch.full((B,), L, dtype=torch.int32, device=dev())
    lse = torch.zeros(B, Hq, device=dev())
    out = qlq.kv_attention(bf16_to_gpu(np.tile(qb, (B, 1, 1))), qlq.QuantizedKV4(both(kc), ks, both(vc), vs), table, lens, page,
                           scale=1.0, lse=lse)
    q64, got, got_lse = bits_to_f64(qb), bits_to_f64(bf16_bits(out)), lse.cpu().numpy().astype(np.float64)
    for h in range(Hq):
        s = k[:L, h // (Hq // Hk)] @ q64[h]
        p = np.exp(s - s.max())
        l64 = s.max() + np.log(p.sum())
        p /= p.sum()
        o64 = p @ v[:L, h // (Hq // Hk)]
        E = U * (3 * (2 * np.abs(s).max() + 56) + L / 32 + 40)
        bound = 2.0 ** -8 * o64 + (2.0 ** -11 + 2 * E) * o64 + L * 2.0 ** -39 * 6              # (v >= 0: S = o)
        over = np.abs(got[:, h] - o64) / bound
        assert over.max() <= 1.0, f"head {h}: {over.max():.2f} times the bound"
        assert np.abs(got_lse[:, h] - l64).max() <= 2 * E + U * abs(l64)


@pytest.mark.parametrize("case", [((1, 1, 1), (40, 20, 90)), ((1, 1), (9000, 700)), ((150, 40), (150, 300)), ((90,), (3000,))])
def test_a_query_with_nan_is_nan_in_its_own_row_alone(case):
    nqs, lens = case
    for Hq, Hk, D in ((4, 2, 64), (4, 1, 128)):
        p = Problem(sum(lens) + D, nqs, lens, Hq, Hk, D, 16, each=False)
        lse0, lse = torch.zeros(p.T, Hq, device=dev()), torch.zeros(p.T, Hq, device=dev())
        out0 = p.run(lse=lse0).clone()
        hit = [(0, 1), (p.T - 1, 3)]
        for t, h in hit:
            p.q[t, h, 5] = float("nan")
        out = p.run(lse=lse)
        for t, h in hit:
            assert bool(torch.isnan(out[t, h]).all()) and bool(torch.isnan(lse[t, h]))
            out[t, h], lse[t, h] = out0[t, h], lse0[t, h]
        assert torch.equal(out, out0) and torch.equal(lse, lse0)


@pytest.mark.parametrize("nqs", [(1,), (3,), (150,)])
def test_a_seen_entry_with_a_nan_scale_shows(nqs):
    for which, D in ((1, 64), (3, 64), (1, 128), (3, 128)):
        p = Problem(3, nqs, (nqs[0] + 100,), 4, 2, D, 16, each=False)
        p.host[which][p.used(0)[50], 1, 1] = 0x7E00
        p.upload()
        out = p.run()
        assert bool(torch.isfinite(out[:, :2].float()).all())                # KV head 0
        bad = torch.isnan(out[:, 2:])
        assert bool(bad.all() if which == 1 else bad[..., 32:64].all() and not bad[..., :32].any())


def test_strided_queries_and_shared_pages():
    p = Problem(11, (1, 1, 1), (200, 150, 90), 8, 2, 128, 16)
    wide = torch.zeros((3, 12 * 128), dtype=torch.bfloat16, device=dev())
    q = wide.as_strided((3, 8, 128), (12 * 128, 128, 1), 0)
    q.copy_(p.q)
    assert torch.equal(qlq.kv_attention(q, p.cache, p.bt, p.sl, 16), p.run())
    t = p.table.copy()
    t[1, :5] = t[0, :5]
    out = qlq.kv_attention(p.q, p.cache, _gpu(t.astype(np.int32), torch.int32), p.sl, 16)
    p.compare(out, None, t, p.lens, what="shared pages")


def test_split_work_repeats_bit_for_bit_and_shares_a_workspace():
    ps = [Problem(12, (1,), (40001,), 7, 1, 64, 256), Problem(13, (1,) * 5, (3000, 10, 500, 1, 2500), 4, 4, 128, 64),
          Problem(24, (333, 50), (900, 2000), 8, 2, 128, 64, each=False), Problem(26, (5, 3), (7000, 300), 6, 3, 192, 32, each=False)]
    want = [p.check(what="once") for p in ps]
    need = [qlq.kv_attention_workspace_bytes(p.T, len(p.lens), p.Hq, p.Hk, p.D, p.q0 is None, 4) for p in ps]
    ws = torch.zeros(max(need), dtype=torch.uint8, device=dev())
    eight = qlq.kv_cache(1024, 2, 64)
    e = lambda **kw: qlq.kv_attention(ps[0].q[:, :4].contiguous(), eight, torch.arange(4, dtype=torch.int32, device=dev())[None],
                                      torch.tensor([900], dtype=torch.int32, device=dev()), 256, **kw)
    e0 = e()
    for _ in range(3):
        for p, w in zip(ps, want):
            assert torch.equal(p.run(), w) and torch.equal(p.run(workspace=ws), w)
            assert not ws[:262144].any(), "arrival counters left at zero"
        assert torch.equal(e(workspace=ws), e0)                               # the 8-bit operator's calls in between


def test_mixed_batch_and_many_sequences():
    Problem(14, (1, 200, 1, 1, 7), (1500, 260, 3, 700, 7), 8, 2, 128, 64, each=False).check(what="mixed")
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 60, size=200)]
    Problem(15, (1,) * 200, lens, 2, 1, 64, 16).check(what="200 sequences")
    nqs = [int(x) for x in rng.integers(0, 4, size=150)]
    Problem(16, nqs, [n + int(e) for n, e in zip(nqs, rng.integers(0, 50, size=150))], 2, 1, 64, 16, each=False).check(
        what="150 sequences of 0 to 3 queries")


@pytest.mark.parametrize("heads", [(34, 1, 128), (72, 1, 64), (130, 2, 96), (128, 1, 192), (1024, 1, 32), (1024, 1024, 32),
                                   (331, 331, 32), (6, 6, 64), (5, 5, 128)])
def test_single_tokens_of_many_heads(heads):
    Hq, Hk, D = heads
    print(f"attention4 heads={heads}", flush=True)
    Problem(Hq + Hk + D, [1] * 4, [0, 1, 65, 200], Hq, Hk, D, 16).check(what=f"{heads}")


@pytest.mark.parametrize("nqs", [(1, 1), (90, 70)])
def test_offsets_beyond_four_gigabytes(nqs):
    Hk, D, page = 8, 256, 256
    pool = (((1 << 33) // (Hk * D)) // page + 3) * page
    small = Problem(20, nqs, (500, 300), 8, Hk, D, page)
    pages = small.pool // page
    big = qlq.QuantizedKV4(*(torch.empty((pool, Hk, D // n), dtype=t, device=dev())
                             for n, t in ((2, torch.uint8), (32, torch.float16)) * 2))
    at = pool - pages * page                           # the sequences' pages at the pool's end
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(big, n)[at:] = getattr(small.cache, n)
    bt = torch.where((small.bt >= 0) & (small.bt < pages), small.bt + at // page, small.bt)
    assert torch.equal(qlq.kv_attention(small.q, big, bt, small.sl, page, q_start=small.q0), small.run())


def test_unwritten_entries_of_a_fresh_cache():
    for n in (1, 70):
        c = qlq.kv_cache(128, 2, 64, bits=4)
        c.v_scales.zero_()
        q = bf16_to_gpu(oracle.f32_to_bf16_bits(np.ones((n, 4, 64), np.float32)))
        lse = torch.zeros(n, 4, device=dev())
        out = qlq.kv_attention(q, c, torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device=dev()),
                               torch.tensor([100], dtype=torch.int32, device=dev()), 32, causal=False, lse=lse,
                               q_start=torch.tensor([0, n], dtype=torch.int32, device=dev()))
        assert not out.any() and torch.allclose(lse, torch.full_like(lse, math.log(100.0)), rtol=1e-6)


def test_two_streams_at_once():
    ps = [Problem(17, (1,), (30000,), 4, 1, 64, 256), Problem(18, (1, 1), (20000, 9000), 4, 1, 64, 256)]
    want = [p.run() for p in ps]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(10):
        for p, w, s in zip(ps, want, streams):
            with torch.cuda.stream(s):
                outs.append((p.run(), w))
    torch.cuda.synchronize()
    for got, w in outs:
        assert torch.equal(got, w)


def test_captured_and_replayed_with_changing_lengths():
    p = Problem(19, (1, 1), (9000, 4000), 4, 1, 64, 256)
    full, short = p.sl.clone(), torch.tensor([33, 4000], dtype=torch.int32, device=dev())
    out, want = torch.empty_like(p.q), p.run().clone()
    p.sl = short
    want_short = p.run().clone()
    p.sl = full.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(out=out)
        graphs.append(g)
    for i in range(6):
        p.sl.copy_(short if i % 3 == 1 else full)
        out.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        w = want_short if i % 3 == 1 else want
        assert torch.equal(out, w) and torch.equal(p.run(), w), i             # eager between the replays


def test_two_graphs_replayed_at_once():
    ps = [Problem(30, (1,), (30000,), 4, 1, 64, 256), Problem(31, (150, 40), (1000, 700), 4, 2, 128, 64, each=False)]
    want, outs, graphs = [p.run().clone() for p in ps], [torch.empty_like(p.q) for p in ps], []
    for p, o in zip(ps, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for p, o, w in zip(ps, outs, want):
            assert torch.equal(o, w) and torch.equal(p.run(), w)


def test_binding_refusals_on_the_gpu():
    p = Problem(21, (1, 1), (20, 30), 4, 2, 64, 16)
    c = p.cache
    bad = [lambda: qlq.kv_attention(p.q, qlq.QuantizedKV(c.k_codes, c.k_scales, c.v_codes, c.v_scales), p.bt, p.sl, 16),
           lambda: qlq.kv_attention(p.q, qlq.kv_cache(64, 2, 96, bits=4), p.bt, p.sl, 16),
           lambda: qlq.kv_attention(p.q, qlq.QuantizedKV4(c.k_codes, c.k_scales, c.v_codes, c.v_scales[:, :, :1]), p.bt, p.sl, 16),
           lambda: qlq.kv_attention(p.q, qlq.QuantizedKV4(c.k_codes, c.k_scales.float(), c.v_codes, c.v_scales), p.bt, p.sl, 16),
           lambda: qlq.kv_attention(p.q, qlq.QuantizedKV4(*(t.cpu() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales))),
                                    p.bt, p.sl, 16),
           lambda: qlq.kv_attention(p.q.float(), c, p.bt, p.sl, 16), lambda: qlq.kv_attention(p.q, c, p.bt.long(), p.sl, 16)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    small = torch.zeros(qlq.kv_attention_workspace_bytes(2, 2, 4, 2, 64, True, 4) - 256, dtype=torch.uint8, device=dev())
    for kw in (dict(page_size=24), dict(page_size=16, window=-1), dict(page_size=16, workspace=small)):
        with pytest.raises(qlq.QlqError):
            qlq.kv_attention(p.q, c, p.bt, p.sl, **kw)


def _seeing(p, b, t, causal, window):
    """The rows of sequence b that see its token t."""
    pos = p.lens[b] - p.nqs[b] + np.arange(p.nqs[b])
    see = (t <= pos) if causal else np.ones(pos.size, bool)
    if window:
        see &= t > pos - window
    return p.starts[b] + np.nonzero(see)[0]


def _check_nan_groups(p, bad, causal=True, window=0, what=""):
    """V scales of (sequence, token, KV head, group) in `bad` become NaN: NaN in those channels of the rows that see the
    token, and everything else as with the finite scales, to its bound."""
    clean, lse, G = p.check(causal=causal, window=window, what=what), torch.zeros(p.T, p.Hq, device=dev()), p.Hq // p.Hk
    want = torch.zeros(clean.shape, dtype=torch.bool)
    for b, t, h, g in bad:
        p.cache.v_scales[int(p.used(b)[t]), h, g] = float("nan")
        want[torch.from_numpy(_seeing(p, b, t, causal, window)), h * G:(h + 1) * G, 32 * g:32 * g + 32] = True
    out = p.run(causal=causal, window=window, lse=lse)
    want = want.to(dev())
    assert torch.equal(torch.isnan(out), want), f"{what}: {int((torch.isnan(out) & ~want).sum())} NaN more, {int((~torch.isnan(out) & want).sum())} fewer"
    p.compare(torch.where(want, clean, out), lse, p.table, p.lens, causal=causal, window=window, what=what)


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 96), (4, 1, 128), (2, 1, 256), (3, 1, 192)])
@pytest.mark.parametrize("case", [((1,), (700,)), ((1, 1, 1), (40, 100, 9000)), ((3,), (500,)), ((150,), (250,))])
def test_groups_beside_a_nan_scale_of_the_heaviest_token(case, heads):
    # the token that outweighs all others has a NaN scale in one group and V scales of 2^6 and more in its others
    (nqs, lens), (Hq, Hk, D) = case, heads
    print(f"attention4 NaN scale of the heaviest token nqs={nqs} heads={heads}", flush=True)
    p = Problem(sum(lens) + D, nqs, lens, Hq, Hk, D, 16, each=False, qgain=4.0)
    q, k, bad = bits_to_f64(p.qb), p.values()[0], []
    for b, n in enumerate(nqs):
        for h in range(Hk):
            t = int(np.argmax(k[p.used(b)[:lens[b] - n + 1], h] @ q[p.starts[b], h * (Hq // Hk)]))
            p.host[3][p.used(b)[t], h] = oracle.fp16_encode((2.0 ** (6 + np.arange(D // 32))).astype(np.float32))
            bad.append((b, t, h, (b + h) % (D // 32)))
    p.upload()
    _check_nan_groups(p, bad, what="heaviest")


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 96), (4, 2, 128), (2, 1, 256), (3, 1, 192), (2, 2, 32)])
@pytest.mark.parametrize("case", [((5,), (40,)), ((4, 1, 9), (300, 1, 80)), ((24,), (5000,)), ((150,), (250,)), ((90, 300), (90, 421))])
def test_a_nan_scale_of_v_stays_with_the_rows_that_see_its_token(case, heads):
    (nqs, lens), (Hq, Hk, D) = case, heads
    print(f"attention4 NaN scales nqs={nqs} heads={heads}", flush=True)
    rng = np.random.default_rng(D + sum(lens))
    for causal, window in ((True, 0), (True, 37), (False, 0)):
        p = Problem(sum(nqs) + D + window, nqs, lens, Hq, Hk, D, 16, each=False)
        bad = []
        for b, (n, L) in enumerate(zip(nqs, lens)):
            # the last token, one between the queries, one that the window hides from the later of them
            for t in {L - 1, L - 1 - n // 2, max(0, L - n - max(window, 30) + 1 + n // 2)}:
                bad.append((b, t, int(rng.integers(Hk)), int(rng.integers(D // 32))))
        _check_nan_groups(p, bad, causal, window, what=f"causal={causal} window={window}")


@pytest.mark.parametrize("heads", [(4, 2, 64), (2, 1, 96), (4, 1, 128), (2, 1, 256), (3, 1, 192), (3, 1, 32)])
def test_small_keys_and_large_queries(heads):
    # K scales down to fp16's smallest, whose products with the codes leave fp16's normal range
    Hq, Hk, D = heads
    print(f"attention4 small keys heads={heads}", flush=True)
    for nqs, lens in (((150,), (250,)), ((3,), (250,))):
        for octaves in (14, 20, 23):
            p = Problem(D + octaves, nqs, lens, Hq, Hk, D, 16, each=False, qgain=2.0 ** octaves)
            s, rng = p.used(0), np.random.default_rng(octaves)
            p.host[0][s], p.host[1][s] = kvcache.kv4_quantize_values(2.0 ** -octaves * rng.standard_normal((s.size, Hk, D)))
            p.upload()
            p.check(what=f"2^-{octaves}")


@pytest.mark.parametrize("heads", [(4, 2, 64), (4, 1, 128), (2, 1, 256), (2, 1, 96), (3, 1, 192)])
def test_keys_beside_one_a_million_times_as_large(heads):
    # Keys of 2^-11 in one tile with a key of 60000 that the last query alone sees.  All of them are code 0.5 of one scale
    # whose bits below the 6th do not fall away by chance, and queries are positive: errors of K add up in every score.
    # The others' scores alone set the bound (A and E of the module's docstring, K's 11 bits among it).
    Hq, Hk, D = heads
    n, L, G = 150, 250, Hq // Hk
    p = Problem(D, (n,), (L,), Hq, Hk, D, 16, each=False, octaves=0)
    s, rng = p.used(0), np.random.default_rng(D)
    p.host[0][s], p.host[1][s] = 0x11, oracle.fp16_encode(np.float32(2.0 ** -10 * (1 + 7 / 1024)))
    p.host[1][s[-1]] = oracle.fp16_encode(np.float32(60000.0))
    p.upload()
    p.qb = oracle.f32_to_bf16_bits((2.0 ** 9 * rng.uniform(1, 2, size=(p.T, Hq, D))).astype(np.float32))
    p.q = bf16_to_gpu(p.qb)
    q, (kv, vv) = bits_to_f64(p.qb), p.values()
    lse = torch.zeros(p.T, Hq, device=dev())
    out = bits_to_f64(bf16_bits(p.run(lse=lse)))[:-1]
    o64, l64, _, S = layer.kv_attention(q, kv, vv, p.table, p.lens, p.page, p.starts)
    ks = np.abs(kv[s[:-1]])
    A = D ** -0.5 * max((np.abs(q[:-1, h]) @ ks[:, h // G].T).max() for h in range(Hq))
    A1 = D ** -0.5 * np.abs(q).max() * ks.sum(-1).max()
    E = U * (42 * A + A1 + 3 * (2 * A + 56) + L / 32 + 40) + 2.0 ** -11 * A
    d = np.abs(lse.cpu().numpy().astype(np.float64) - l64)[:-1] - (2 * E + U * np.abs(l64[:-1]))
    assert d.max() <= 0, f"lse {d.max():.3e} beyond the bound"
    over = np.abs(out - o64[:-1]) - (2.0 ** -8 * np.abs(o64[:-1]) + S[:-1] * (2.0 ** -10 + 2 * E) + L * 2.0 ** -31 * np.abs(vv[s]).max())
    assert np.max(over) <= 0, f"{np.max(over):.3e} beyond the bound"
